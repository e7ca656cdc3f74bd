"""Which form a call of query chunks takes, and what workspace it asks for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from test_gpu_extend import Batch, check_sequences


@pytest.mark.parametrize("order", [1, -1])
def test_a_long_context_beside_a_long_chunk_is_split(order):
    """One long prompt chunk and one row over a far longer context: the row's
    keys go over many CTAs, which only a plan does."""
    new, lens = [2048, 1][::order], [2048, 60000][::order]
    b = Batch(new, lens, 32, 32, 64, seed=1)
    planned = b.run(True)
    K.kvs_pool_set_test_flags(b.pool, 0)
    before = K.kvs_launch_count()
    out = b.run(True)
    assert K.kvs_launch_count() > before + 1
    assert torch.equal(out, planned)
    check_sequences(b, out, [new.index(1)], True)


def test_short_rows_over_one_prefix_beside_a_long_chunk_are_shared():
    """Many short rows over one long prefix and a chunk that makes up the mean
    length: the prefix is read once, so the plan is taken."""
    new, lens = [2] * 15 + [2600], [8192 + 2] * 15 + [2600]
    b = Batch(new, lens, 32, 2, 64, prefix=[8192, 0], groups=[0] * 15 + [1], seed=2)
    planned = b.run(True)
    K.kvs_pool_set_test_flags(b.pool, 0)
    before = K.kvs_launch_count()
    assert torch.equal(b.run(True), planned)
    assert K.kvs_launch_count() > before + 1
    check_sequences(b, planned, [0, 14], True)
