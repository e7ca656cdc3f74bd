"""The operators on new tokens take tensors of the current device alone (their
pool is checked against it too).  Stand-ins for tensors of another device: no
GPU is needed to ask."""
import pytest

torch = pytest.importorskip("torch")

from shared_paged_kv_gb300 import kvs as K


class On:
    """What the binding asks a contiguous CUDA tensor of device `at`."""

    is_cuda = True

    def __init__(self, at, dtype, *shape):
        self.at, self.dtype, self.shape = at, dtype, shape

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return 1

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("current, at", [(0, 0), (1, 1), (0, 1), (1, 0)])
def test_tensors_of_another_device_are_refused(monkeypatch, current, at):
    monkeypatch.setattr(K, "_cur_dev", lambda: current)
    calls = [lambda: K._rows(On(at, torch.bfloat16, 4, 2, 64), 4, 2, 64, "q"), lambda: K._ints(On(at, torch.int32, 5), 5, "tok_off"),
             lambda: K._table(On(at, torch.int32, 3, 7), 3, 7), lambda: K._positions(On(at, torch.int32, 3, 4), 3, 4),
             lambda: K._ws(On(at, torch.uint8, 64))]
    for call in calls:
        if current == at:
            call()
        else:
            with pytest.raises(ValueError):
                call()
