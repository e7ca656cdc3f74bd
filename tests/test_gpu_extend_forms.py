"""Which form a call of query chunks takes, and what workspace it asks for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from test_gpu_extend import DEV, Batch, check_sequences


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


def plan_counts(ws):
    """(items, units, part rows) of the plan in ws, from its header."""
    h = ws[:64].cpu().numpy().view(np.int32)
    return int(h[7]), int(h[9]), int(h[10])


@pytest.mark.parametrize("n, hq, hkv, d", [(128, 8, 8, 64), (700, 4, 4, 64), (40, 32, 32, 128), (90, 14, 7, 128)])
def test_a_long_context_among_many_short_ones_is_split(n, hq, hkv, d):
    """More units than the device needs, one of them far longer than the rest:
    its keys go over many CTAs, the others' do not."""
    r = np.random.default_rng(n)
    new = r.integers(1, 3, n)
    lens = new + r.integers(0, 300, n)
    lens[n // 3] = 40000
    b = Batch(new, lens, hq, hkv, d, seed=n)
    ws = b.ws()
    out = b.run(True, ws=ws)
    items, units, parts = plan_counts(ws)
    # pieces of at most half an SM's mean load of key tiles (of 128)
    tiles = -(-lens // 128)
    load = -(-int(tiles.sum()) * hkv // torch.cuda.get_device_properties(DEV).multi_processor_count)
    pieces = -(-int(tiles.max()) // max(2, (load + 1) // 2))
    assert units == n and pieces > 4 and items >= n - 1 + pieces
    assert 0 < parts <= 2 * (hq // hkv) * 2 * (items - n)      # at most two rows a unit; a cut one has two pieces or more
    check_sequences(b, out, [n // 3, 0, n - 1, n // 3 + 1], True)
    assert torch.equal(out, b.run(True, ws=ws))


def test_equal_contexts_that_fill_the_device_are_not_split():
    b = Batch([1] * 128, [1000 + 3 * i for i in range(128)], 8, 8, 64, seed=2)
    ws = b.ws()
    b.run(True, ws=ws)
    assert plan_counts(ws) == (128, 128, 0)


@pytest.mark.parametrize("hq, hkv, rows", [(8, 8, 20000), (32, 2, 10000)])
def test_a_chunk_longer_than_its_sequence(hq, hkv, rows):
    """One sequence, far more rows than it has tokens: all but the last rows
    see nothing, and the few that see keys are the longest units."""
    b = Batch([rows], [900], hq, hkv, 64, seed=3)
    out = b.run(True)
    assert (out[:rows - 900] == 0).all()
    b.q, b.T, b.off, b.new = b.q[rows - 900:], 900, np.array([0, 900]), np.array([900])
    check_sequences(b, out[rows - 900:], [0], True)
