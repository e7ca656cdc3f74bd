"""Arguments of the operators on new tokens: empty steps, tensors laid out for
another shape, workspaces that are not on the GPU, scales at the end of the
range."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
import harness as H
from test_gpu_append import Case, randn
from test_gpu_extend import Batch

DEV = H.DEV


def test_an_empty_step_with_queries_does_nothing():
    """No new token of any sequence: every call of the step is a no-op, also
    with (empty) queries beside the rows."""
    c = Case([0, 0], [5, 40], 2, 128)
    before = [s.clone() for s in c.slabs]
    k, q = randn(1, 0, 2, 128), randn(2, 0, 8, 128)
    c.append(k, k, rope=K.RopeAxes(1e6, (64,)), q=q, n_q_heads=8, q_out=torch.empty_like(q))
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    c.append(k, k, rope=K.RopeAxes(1e6, (16, 24, 24)), pos=none, q=q, n_q_heads=8, q_out=torch.empty_like(q))
    c.gather(k, k.clone())
    K.kvs_rope_apply(q, torch.empty(1, 0, dtype=torch.int32, device=DEV), K.RopeAxes(1e6, (64,)), torch.empty_like(q), 0, 8, 128)
    off, tab, mb, lens, n = c.args()
    ws = H.workspace(K.kvs_extend_workspace_size(c.pool, 0, n, mb, 8))
    K.kvs_extend_attn(c.pool, 0, q, 0, off, 8, tab, mb, lens, n, True, 1.0, torch.empty_like(q), ws)
    assert K.kvs_pool_check(c.pool) == 0
    assert torch.equal(before[0], c.slabs[0]) and torch.equal(before[1], c.slabs[1])


def test_queries_and_their_result_go_together_in_a_step_with_rows():
    c = Case([2], [5], 2, 128)
    k, q = randn(1, 2, 2, 128), randn(2, 2, 8, 128)
    for kw in (dict(q=q, n_q_heads=8), dict(q_out=q, n_q_heads=8), dict(n_q_heads=8),
               dict(rope=K.RopeAxes(1e6, (16, 24, 24)))):
        with pytest.raises((K.KvsError, ValueError)):
            c.append(k, k, **kw)


def test_positions_of_another_length_are_refused():
    """Positions are [axes][n_tokens]: of a longer padded batch the second axis
    would be read at the wrong place."""
    c = Case([4, 3], [0, 9], 2, 128)
    k, v = randn(1, 7, 2, 128), randn(2, 7, 2, 128)
    rope = K.RopeAxes(1e6, (16, 24, 24))
    pos = H.i32(np.arange(3 * 9).reshape(3, 9))
    x = randn(3, 7, 4, 128)
    for bad in (pos, pos.flatten(), pos[:2], H.i32(np.arange(21).reshape(7, 3))):
        with pytest.raises(ValueError):
            c.append(k, v, rope=rope, pos=bad)
        with pytest.raises(ValueError):
            K.kvs_rope_apply(x, bad, rope, torch.empty_like(x), 7, 4, 128)
    good = pos[:, :7].contiguous()
    a, b = torch.empty_like(x), torch.empty_like(x)
    K.kvs_rope_apply(x, good, rope, a, 7, 4, 128)
    K.kvs_rope_apply(x, good.flatten(), rope, b, 7, 4, 128)
    assert torch.equal(a, b)
    c.append(k, v, rope=rope, pos=good)
    # on one axis a longer tensor begins with the same positions
    one = K.RopeAxes(1e6, (64,))
    K.kvs_rope_apply(x, pos[0, :7].contiguous(), one, a, 7, 4, 128)
    K.kvs_rope_apply(x, pos[:1], one, b, 7, 4, 128)
    assert torch.equal(a, b)
    assert K.kvs_pool_check(c.pool) == 0


def test_tables_of_another_width_are_refused():
    """A table is [n_seq][max_blocks]: with wider rows the second sequence's
    blocks would be read from the first one's."""
    c = Case([4, 3], [0, 9], 2, 128)
    k, v, q = randn(1, 7, 2, 128), randn(2, 7, 2, 128), randn(3, 7, 8, 128)
    off, tab, mb, lens, n = c.args()
    assert mb > 1
    ws = H.workspace(K.kvs_extend_workspace_size(c.pool, 7, n, mb, 8))
    out = torch.empty_like(q)
    for m in (mb - 1, mb + 1):
        with pytest.raises(ValueError):
            K.kvs_append(c.pool, 0, k, v, 7, off, tab, m, lens, n)
        with pytest.raises(ValueError):
            K.kvs_gather(c.pool, 0, 7, off, tab, m, lens, n, k, v)
        with pytest.raises(ValueError):
            K.kvs_extend_plan(c.pool, 7, off, 8, tab, m, lens, n, True, ws)
        for f in (K.kvs_extend_attn, K.kvs_extend_attn_planned):
            with pytest.raises(ValueError):
                f(c.pool, 0, q, 7, off, 8, tab, m, lens, n, True, 1.0, out, ws)
    with pytest.raises(ValueError):                          # one row does not go on in the next
        K.kvs_append(c.pool, 0, k, v, 7, off, tab, 2 * mb, lens, 1)
    K.kvs_gather(c.pool, 0, 4, off, tab, mb - 1, lens, 1, k[:4].clone(), v[:4].clone())   # a row may be longer than asked
    wide = torch.cat([tab, torch.full_like(tab, -1)])       # more sequences than the call's: the first rows
    K.kvs_append(c.pool, 0, k, v, 7, off, wide, mb, lens, n)
    K.kvs_append(c.pool, 0, k, v, 7, off, tab.flatten(), mb, lens, n)
    assert K.kvs_pool_check(c.pool) == 0


def test_a_workspace_that_is_not_on_the_gpu_is_refused():
    b = Batch([4, 9], [70, 65], 8, 2, 64)
    off, tab, lens = b.dev()
    n = b.ws().numel()
    out = torch.empty_like(b.q)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(n, 2, dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            K.kvs_extend_plan(b.pool, b.T, off, 8, tab, b.mb, lens, b.n, True, bad)
        for f in (K.kvs_extend_attn, K.kvs_extend_attn_planned):
            with pytest.raises(ValueError):
                f(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, bad)
    wide = torch.empty(-(-n // 4), dtype=torch.int32, device=DEV)     # any type: its bytes count
    K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, wide)
    assert torch.equal(out, b.run(True))


def test_scales_at_the_end_of_the_range():
    """The exponent's base change must not leave the float32 range: a scale
    that does is refused, the largest that does not gives finite results."""
    b = Batch([3], [3], 8, 2, 64)
    off, tab, lens = b.dev()
    q, out = torch.zeros_like(b.q), torch.empty_like(b.q)
    ws = b.ws()
    for scale in (3e38, 2.4e38):
        with pytest.raises(K.KvsError):
            K.kvs_extend_attn(b.pool, 0, q, b.T, off, 8, tab, b.mb, lens, b.n, True, scale, out, ws)
    K.kvs_extend_attn(b.pool, 0, q, b.T, off, 8, tab, b.mb, lens, b.n, True, 2.3e38, out, ws)
    assert K.kvs_pool_check(b.pool) == 0
    assert torch.isfinite(out.float()).all() and (out[0, 0] == b.v[b.table[0, 0], 0, 0]).all()
