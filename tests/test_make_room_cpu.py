"""What the operators that make room refuse before anything reaches a GPU: by the binding (tensors of another device,
type or shape; stand-ins, no GPU is needed to ask) and by the library (no pool)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from shared_paged_kv_gb300 import kvs as K
from test_binding_devices import On


class Desc:
    num_kv_heads, head_dim, block_tokens, capacity_blocks = 2, 64, 16, 8


class FakePool:
    handle, desc = None, Desc


@pytest.mark.parametrize("current, at", [(0, 0), (1, 1), (0, 1), (1, 0)])
def test_tensors_of_another_device_are_refused(monkeypatch, current, at):
    monkeypatch.setattr(K, "_cur_dev", lambda: current)
    for call in (lambda: K._floats(On(at, torch.float32, 5), 5, "out"), lambda: K._offsets(On(at, torch.int64, 5), 5, "idx_off"),
                 lambda: K._mass(On(at, torch.float32, 3, 64), FakePool, 3, 4, "mass")):
        if current == at:
            call()
        else:
            with pytest.raises(ValueError):
                call()


def test_types_and_shapes(monkeypatch):
    monkeypatch.setattr(K, "_cur_dev", lambda: 0)
    assert K._mass(On(0, torch.float32, 192), FakePool, 3, 4, "mass") == 4096         # one dimension
    assert K._mass(On(0, torch.float32, 5, 64), FakePool, 3, 4, "mass") == 4096       # more sequences
    assert K._mass(None, FakePool, 3, 4, "mass_in") is None and K._floats(None, 3, "x") is None
    for bad in (lambda: K._mass(On(0, torch.float32, 3, 65), FakePool, 3, 4, "mass"),
                lambda: K._mass(On(0, torch.float32, 2, 64), FakePool, 3, 4, "mass"),
                lambda: K._mass(On(0, torch.float64, 3, 64), FakePool, 3, 4, "mass"),
                lambda: K._floats(On(0, torch.float32, 4), 5, "out"), lambda: K._floats(On(0, torch.bfloat16, 5), 5, "out"),
                lambda: K._offsets(On(0, torch.int32, 5), 5, "idx_off"), lambda: K._offsets(On(0, torch.int64, 4), 5, "idx_off")):
        with pytest.raises(ValueError):
            bad()


def test_no_pool():
    import __graft_entry__ as g
    g.build()
    lib = K.load()
    n = ctypes.c_size_t()
    assert lib.kvs_keep_heavy(None, None, None, 1, 1, None, 0, 0, None, None, None) == K.KVS_ERR_INVALID_ARG
    assert lib.kvs_compact(None, None, 1, None, 1, None, None, None, None, None, None, None, 0, None) == K.KVS_ERR_INVALID_ARG
    for fn in (lib.kvs_decode_attn_mass, lib.kvs_decode_attn_mx4):
        assert fn(None, 0, None, 8, None, 1, None, 1, 0.1, None, None, 1.0, None, None, 0, None) == K.KVS_ERR_INVALID_ARG
    assert lib.kvs_extend_mass(None, 0, None, 64, None, 1, 8, None, 1, None, 1, 1, 0.1, None, 1.0, None, None, 0, None) == K.KVS_ERR_INVALID_ARG
    assert lib.kvs_extend_mass_workspace_size(None, 1, 1, 1, 8, ctypes.byref(n)) == K.KVS_ERR_INVALID_ARG
    out, arr = ctypes.c_void_p(), (ctypes.c_void_p * 1)(16)
    for desc, st in ((K.PoolDesc(1, 2, 64, 64, K.KVS_DTYPE_MX4, 8, 0, 4), K.KVS_ERR_UNSUPPORTED),
                     (K.PoolDesc(1, 2, 128, 16, K.KVS_DTYPE_MX4, 8, 0, 4), K.KVS_ERR_UNSUPPORTED),
                     (K.PoolDesc(1, 2, 128, 64, K.KVS_DTYPE_MX4, 8, 4, 4), K.KVS_ERR_UNSUPPORTED),
                     (K.PoolDesc(1, 2, 128, 64, K.KVS_DTYPE_MX4, 8, 0, 4), K.KVS_ERR_INVALID_ARG)):   # no scales
        assert lib.kvs_pool_create(ctypes.byref(desc), arr, arr, None, None, None, None, ctypes.byref(out)) == st
