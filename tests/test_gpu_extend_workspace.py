"""The workspace of chunk attention: sized for a step, it serves every smaller
one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from test_gpu_extend import Batch, DEV, check_sequences


def pool(hkv, d=128, max_seqs=4096):
    slab = [torch.zeros(2, hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    return K.kvs_pool_create(1, hkv, d, 16, K.KVS_DTYPE_BF16, 2, max_seqs, [slab[0]], [slab[1]])


@pytest.mark.parametrize("hkv, hq", [(32, 32), (8, 40), (2, 16), (1, 12), (8, 8)])
def test_a_larger_step_needs_no_less(hkv, hq):
    p = pool(hkv)
    tokens = sorted({1, 2, 15, 100, 255, 256, 257, 1000, 4096, 8192, 16384, 16385, 30000, 65536, 65537, 200000,
                     (1 << 19) // hq, (1 << 19) // hq + 1, (1 << 19) // hq - 1})
    seqs, blocks = [1, 2, 3, 32, 33, 600, 4096], [1, 8, 96, 97, 500, 4096]
    size = np.array([[[K.kvs_extend_workspace_size(p, t, n, b, hq) for b in blocks] for n in seqs] for t in tokens])
    for axis in range(3):
        assert (np.diff(size, axis=axis) >= 0).all(), "tokens sequences blocks".split()[axis]


def test_one_buffer_for_every_step():
    """Sized for a step above the rows that are ever split or shared, used by
    one at that bound and by small ones, shared and split."""
    hq = 32
    big = Batch([4100, 4200, 4000, 4085], [4100, 4200, 4000, 4085], hq, 4, 64, seed=3)
    assert big.T * hq > 1 << 19
    ws = torch.full((K.kvs_extend_workspace_size(big.pool, big.T, big.n, big.mb + 200, hq),), 255, dtype=torch.uint8, device=DEV)
    for b in (Batch([4096, 4096, 4096, 4096], [4096] * 4, hq, 4, 64, prefix=64, seed=4),   # 2^19 rows
              Batch([3, 1, 2, 2], [3000, 2500, 1300, 900], hq, 4, 64, seed=5),
              Batch([3, 1, 2, 2], [1000 + 3, 1001, 1100, 1030], hq, 4, 64, prefix=1000 // 16 * 16, seed=6),
              Batch([70], [5000], hq, 4, 64, seed=7)):
        out = b.run(True, ws=ws)
        if b.T < 100:
            check_sequences(b, out, range(b.n), True)
        else:
            assert torch.equal(out, b.run(True))


def test_a_call_without_a_plan_needs_no_workspace():
    b = Batch([4, 9], [70, 65], 8, 2, 64)
    K.kvs_pool_set_test_flags(b.pool, 0)
    want = b.run(True)
    off, tab, lens = b.dev()
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(32, dtype=torch.uint8, device=DEV)):
        out = torch.full_like(want, 7.0)
        K.kvs_extend_plan(b.pool, b.T, off, 8, tab, b.mb, lens, b.n, True, ws)
        K.kvs_extend_attn_planned(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, ws)
        assert torch.equal(out, want)
        out.fill_(7.0)
        K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, ws)
        assert torch.equal(out, want)
    K.kvs_pool_set_test_flags(b.pool, K.KVS_TEST_EXTEND_PLANNED)
    for ws in (None, torch.empty(32, dtype=torch.uint8, device=DEV)):
        with pytest.raises(K.KvsError):
            K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, torch.empty_like(want), ws)
        with pytest.raises(K.KvsError):
            K.kvs_extend_attn_planned(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, torch.empty_like(want), ws)
    assert K.kvs_pool_check(b.pool) == 0
