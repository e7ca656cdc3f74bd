"""GPU rotary positions, rotated append and read-back against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from oracle import extend as OE, q4 as OQ
import harness as H

DEV = H.DEV
SECTIONS = {(64, 1): (32,), (64, 2): (16, 16), (64, 3): (8, 12, 12), (128, 1): (64,), (128, 2): (32, 32),
            (128, 3): (16, 24, 24)}


def randn(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def assert_rotated(got, exp):
    """Half a bf16 step of the result (2^-8 relative), plus 2^-20 of the
    pair's norm for float32: the angle's reduction and conversion (2 pi 2^-25
    absolute), sincospif and the two products and their sum (2^-24 each, a few
    times) stay below it."""
    h = exp.shape[-1] // 2
    r = np.sqrt(exp[..., :h] ** 2 + exp[..., h:] ** 2)
    tol = 2.0 ** -8 * np.abs(exp) + 2.0 ** -20 * 1.01 * np.concatenate([r, r], -1)
    bad = np.abs(got - exp) > tol
    assert not bad.any(), f"{bad.sum()} off, most {np.abs(got - exp).max():.3e}"


# ---------------------------------------------------------- rope_apply ----
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("axes", [1, 2, 3])
@pytest.mark.parametrize("tokens, heads", [(1, 1), (7, 5), (33, 16), (700, 3)])
@pytest.mark.parametrize("own", [False, True])
def test_rope_apply(d, axes, tokens, heads, own):
    x = randn(tokens + heads, tokens, heads, d)
    r = np.random.default_rng(d + axes)
    pos = r.integers(-(1 << 31), 1 << 31, (axes, tokens))
    pos[:, : tokens // 2] = r.integers(0, 200000, (axes, tokens // 2))
    sec = SECTIONS[d, axes]
    out = torch.full_like(x, float("nan"))
    K.kvs_rope_apply(x, H.i32(pos), K.RopeAxes(1e6, sec, own), out, tokens, heads, d)
    exp = OE.rotate_axes(f64(x), pos, 1e6, sec, own)
    # the frequency is held to 2^-53 of itself (host fp64): 2^31 positions on
    # at most 1/(2 pi) turns each are off by 2^31 2^-53 radians, below the tolerance's 2^-20
    assert_rotated(f64(out), exp)


@pytest.mark.parametrize("n_axes, sec", [(3, (64, 0, 0)), (3, (0, 0, 64)), (2, (63, 1)), (3, (0, 32, 32))])
def test_rope_apply_uneven_sections(n_axes, sec):
    x = randn(3, 9, 2, 128)
    pos = np.random.default_rng(5).integers(0, 5000, (n_axes, 9))
    for own in (False, True):
        out = torch.empty_like(x)
        K.kvs_rope_apply(x, H.i32(pos), K.RopeAxes(1e4, sec, own), out, 9, 2, 128)
        assert_rotated(f64(out), OE.rotate_axes(f64(x), pos, 1e4, sec, own))


def test_rope_apply_views_in_place_and_back():
    """A head range of a projection's rows, rotated in place: the rest of the
    rows stays; rotating back gives the input to two roundings."""
    tokens, d = 400, 128
    rows = randn(1, tokens, 9, d)
    before = rows.clone()
    pos = np.random.default_rng(6).integers(0, 90000, (3, tokens))
    ax = K.RopeAxes(1e6, SECTIONS[d, 3])
    view = rows[:, 2:7]
    K.kvs_rope_apply(view, H.i32(pos), ax, view, tokens, 5, d)
    assert torch.equal(rows[:, :2], before[:, :2]) and torch.equal(rows[:, 7:], before[:, 7:])
    assert_rotated(f64(view), OE.rotate_axes(f64(before[:, 2:7]), pos, 1e6, SECTIONS[d, 3]))
    once = view.clone()
    K.kvs_rope_apply(view, H.i32(pos), ax, view, tokens, 5, d, inverse=True)
    assert_rotated(f64(view), OE.rotate_axes(f64(once), pos, 1e6, SECTIONS[d, 3], inverse=True))


def test_rope_apply_leaves_rows_behind_the_last_token():
    x, out = randn(2, 20, 4, 64), torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    K.kvs_rope_apply(x, H.i32(np.arange(13)[None]), K.RopeAxes(1e4, (32,)), out, 13, 4, 64)
    assert (out[13:] == 7).all() and (out[:13] != 7).any()


# -------------------------------------------------------------- append ----
class Case:
    def __init__(self, new, ctx, hkv, d, q4=False, pad=0, seed=0, extra_blocks=3):
        self.new, self.ctx = np.array(new), np.array(ctx)
        self.n = len(new)
        self.B = 256 if q4 else 16
        self.lens = self.ctx + self.new
        self.off = np.concatenate([[0], np.cumsum(self.new)])
        self.tokens = int(self.off[-1]) + pad
        self.mb = int(-(-max(self.lens.max(), 1) // self.B)) + 1
        r = np.random.default_rng(seed)
        need = -(-self.lens // self.B)
        self.cap = int(need.sum()) + extra_blocks
        ids = r.permutation(self.cap)
        self.table = np.full((self.n, self.mb), -1)
        k = 0
        for a in range(self.n):
            self.table[a, :need[a]] = ids[k:k + need[a]]
            k += need[a]
        self.hkv, self.d, self.q4 = hkv, d, q4
        if q4:
            g = torch.Generator(device=DEV).manual_seed(seed)
            u8 = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
            self.slabs = [u8(self.cap, hkv, 256, d // 2), u8(self.cap, hkv, 256, d // 2),
                          randn(seed + 1, self.cap, hkv, 256, d // 64, 2).to(torch.float16),
                          randn(seed + 2, self.cap, hkv, 256, d // 64, 2).to(torch.float16)]
            self.pool = K.kvs_pool_create(1, hkv, d, 256, K.KVS_DTYPE_Q4G64, self.cap, max(self.n, 1), [self.slabs[0]],
                                          [self.slabs[1]], [self.slabs[2]], [self.slabs[3]])
        else:
            self.slabs = [randn(seed + 1, self.cap, hkv, 16, d), randn(seed + 2, self.cap, hkv, 16, d)]
            self.pool = K.kvs_pool_create(1, hkv, d, 16, K.KVS_DTYPE_BF16, self.cap, max(self.n, 1), [self.slabs[0]],
                                          [self.slabs[1]])

    def args(self):
        return H.i32(self.off), H.i32(self.table), self.mb, H.i32(self.lens), self.n

    def append(self, k, v, **kw):
        off, tab, mb, lens, n = self.args()
        K.kvs_append(self.pool, 0, k, v, self.tokens, off, tab, mb, lens, n, **kw)

    def gather(self, k_out, v_out):
        off, tab, mb, lens, n = self.args()
        K.kvs_gather(self.pool, 0, self.tokens, off, tab, mb, lens, n, k_out, v_out)

    def places(self):
        return OE.places(self.off, self.lens, self.table, self.B)


BATCHES = [
    ([1], [0]), ([1, 1, 1], [15, 16, 31]), ([0, 3, 0, 0, 5], [4, 40, 0, 9, 250]), ([17, 1, 33], [7, 0, 300]),
    ([1] * 40, list(range(0, 400, 10))), ([150, 0, 260], [3, 0, 100]),
]


@pytest.mark.parametrize("new, ctx", BATCHES)
@pytest.mark.parametrize("d, hkv, hq", [(64, 2, 8), (128, 8, 40), (128, 1, 0), (128, 5, 5)])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_append_bf16(new, ctx, d, hkv, hq, axes):
    c = Case(new, ctx, hkv, d, pad=2, seed=len(new) + d)
    k, v = randn(11, c.tokens, hkv, d), randn(12, c.tokens, hkv, d)
    q = randn(13, c.tokens, hq, d) if hq else None
    q_out = torch.full_like(q, 5.0) if hq else None
    before = [s.clone() for s in c.slabs]
    sec = SECTIONS[d, axes] if axes else None
    pl = c.places()
    pos = np.zeros((max(axes, 1), c.tokens), np.int64)
    for t, (_, p, _, _) in pl.items():
        pos[:, t] = p
    kw = {}
    if axes == 3:
        pos = np.random.default_rng(3).integers(0, 70000, (3, c.tokens))
        kw["pos"] = H.i32(pos)
    c.append(k, v, rope=K.RopeAxes(1e6, sec) if axes else None, q=q, n_q_heads=hq, q_out=q_out, **kw)
    assert K.kvs_pool_check(c.pool) == 0
    rot = lambda x: OE.rotate_axes(f64(x), pos, 1e6, sec) if axes else f64(x)  # noqa: E731
    ek = rot(k)
    got_k, got_v = f64(c.slabs[0]), f64(c.slabs[1])
    wk, wv = f64(before[0]), f64(before[1])
    rows = sorted(pl)
    blk, at = np.array([pl[t][2] for t in rows], int), np.array([pl[t][3] for t in rows], int)
    assert_rotated(got_k[blk, :, at], ek[rows])
    wk[blk, :, at] = got_k[blk, :, at]
    wv[blk, :, at] = f64(v)[rows]
    np.testing.assert_array_equal(got_k, wk)      # nothing else was written
    np.testing.assert_array_equal(got_v, wv)
    if hq:
        assert_rotated(f64(q_out)[rows], rot(q)[rows])
        assert (q_out[c.tokens - 2:] == 5).all()  # rows of no sequence
    # and the way back
    k2, v2 = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    c.gather(k2, v2)
    np.testing.assert_array_equal(f64(k2)[rows], got_k[blk, :, at])
    assert torch.equal(v2[rows], v[rows]) and (k2[c.tokens - 2:] == 3).all() and (v2[c.tokens - 2:] == 3).all()
    assert K.kvs_pool_check(c.pool) == 0


def test_append_special_values_pass_through():
    """Values are moved, not multiplied: infinities, NaN and -0 arrive."""
    c = Case([3], [0], 2, 64)
    v = randn(1, 3, 2, 64)
    v[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0], dtype=torch.bfloat16, device=DEV)
    k = v.clone()
    c.append(k, v)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    c.gather(k2, v2)
    assert torch.equal(v2.view(torch.int16), v.view(torch.int16)) and torch.equal(k2.view(torch.int16), k.view(torch.int16))


def test_append_rows_of_one_projection():
    """Queries, keys and values side by side in the rows of one tensor."""
    hq, hkv, d = 16, 2, 128
    c = Case([5, 1, 30], [0, 77, 12], hkv, d)
    qkv = randn(4, c.tokens, hq + 2 * hkv, d)
    q_out = torch.empty(c.tokens, hq, d, dtype=torch.bfloat16, device=DEV)
    ax = K.RopeAxes(1e6, (64,))
    c.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rope=ax, q=qkv[:, :hq], n_q_heads=hq, q_out=q_out)
    a = [s.clone() for s in c.slabs]
    c.append(qkv[:, hq:hq + hkv].contiguous(), qkv[:, hq + hkv:].contiguous(), rope=ax)
    assert torch.equal(a[0], c.slabs[0]) and torch.equal(a[1], c.slabs[1])
    pos = np.array([[c.places()[t][1] for t in range(c.tokens)]])
    assert_rotated(f64(q_out), OE.rotate_axes(f64(qkv[:, :hq]), pos, 1e6, (64,)))
    q = qkv[:, :hq].contiguous()   # in place
    c.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rope=ax, q=q, n_q_heads=hq, q_out=q)
    assert torch.equal(q, q_out)


@pytest.mark.parametrize("new, ctx", [([1] * 12, list(range(0, 3000, 250))), ([257, 0, 33, 700], [0, 5, 255, 300])])
@pytest.mark.parametrize("axes", [0, 1])
def test_append_q4_is_the_quantiser(new, ctx, axes):
    """Codes, scales and biases are those of kvs_quantize_q4 on the values that
    a bf16 pool would hold, bit for bit; the read-back is scale * code + bias."""
    hkv, d = 4, 128
    c, b = Case(new, ctx, hkv, d, q4=True, pad=1), Case(new, ctx, hkv, d, pad=1)
    k, v = randn(21, c.tokens, hkv, d), randn(22, c.tokens, hkv, d)
    v[0, 0, :64] = 0.5                             # a constant group
    rope = K.RopeAxes(1e6, (64,)) if axes else None
    before = [s.clone() for s in c.slabs]
    c.append(k, v, rope=rope)
    b.append(k, v, rope=rope)
    assert K.kvs_pool_check(c.pool) == 0
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    b.gather(kb, vb)
    pl = c.places()
    rows = sorted(pl)
    n = len(rows)
    # the rows as whole blocks of a pool of their own, quantised there
    nb = -(-n // 256)
    src = lambda x: torch.cat([x[rows], torch.zeros(nb * 256 - n, hkv, d, dtype=x.dtype, device=DEV)]).view(nb, 256, hkv, d).transpose(1, 2).contiguous()  # noqa: E731,E501
    s2 = [torch.zeros(nb, hkv, 256, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
         [torch.zeros(nb, hkv, 256, 2, 2, dtype=torch.float16, device=DEV) for _ in range(2)]
    p2 = K.kvs_pool_create(1, hkv, d, 256, K.KVS_DTYPE_Q4G64, nb, 1, [s2[0]], [s2[1]], [s2[2]], [s2[3]])
    K.kvs_quantize_q4(p2, 0, src(kb), src(vb), H.i32(np.arange(nb)), nb)
    blk, at = np.array([pl[t][2] for t in rows]), np.array([pl[t][3] for t in rows])
    for i in range(4):
        want = before[i].cpu().numpy()
        flat = s2[i].transpose(1, 2).reshape(nb * 256, *s2[i].shape[1:2], *s2[i].shape[3:])[:n].cpu().numpy()
        want[blk, :, at] = flat
        np.testing.assert_array_equal(c.slabs[i].cpu().numpy().view(np.uint8), want.view(np.uint8))
    k2, v2 = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    c.gather(k2, v2)
    assert (k2[-1] == 3).all() and (v2[-1] == 3).all()
    code, sb = c.slabs[1].cpu().numpy()[blk, :, at], c.slabs[3].cpu().numpy()[blk, :, at].astype(np.float64)
    val = np.stack([code & 15, code >> 4], -1).reshape(n, hkv, 2, 64) * sb[..., 0:1] + sb[..., 1:2]
    exp = torch.from_numpy(val.reshape(n, hkv, d).astype(np.float32)).to(torch.bfloat16)   # exact in float32 or one rounding
    got = v2[rows].cpu()
    assert (f64(got) - val.reshape(n, hkv, d) <= 2.0 ** -8 * np.abs(val.reshape(n, hkv, d)) + 1e-30).all()
    assert (got != exp).float().mean() < 1e-3


def test_append_and_gather_report_bad_places():
    """A place past the table, a negative one, and bad block ids set their
    flags and drop the key and value alone; queries are still rotated."""
    for change, flag in [("past", K.KVS_DEVERR_SEQ_LEN), ("negative", K.KVS_DEVERR_SEQ_LEN),
                         ("unmapped", K.KVS_DEVERR_BLOCK_ID), ("beyond", K.KVS_DEVERR_BLOCK_ID)]:
        c = Case([4, 2], [20, 3], 2, 64)
        if change == "past":
            c.lens[0] = c.mb * 16 + 4
        elif change == "negative":
            c.lens[0] = 0
        elif change == "unmapped":
            c.table[0, 1] = -1
        else:
            c.table[0, 1] = c.cap
        k, v, q = randn(1, 6, 2, 64), randn(2, 6, 2, 64), randn(3, 6, 4, 64)
        before = c.slabs[0].clone()
        q_out = torch.full_like(q, float("nan"))
        c.append(k, v, rope=K.RopeAxes(1e4, (32,)), q=q, n_q_heads=4, q_out=q_out)
        assert K.kvs_pool_check(c.pool) == flag, change
        changed = (c.slabs[0] != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [c.table[1, 0]], change
        assert torch.isfinite(q_out.float()).all()
        k2 = torch.full_like(k, 3.0)
        c.gather(k2, k2.clone())
        assert K.kvs_pool_check(c.pool) == flag, change
        assert (k2[:4] == 3).all() and (k2[4:] != 3).any(), change


def test_append_refusals():
    c = Case([2], [0], 2, 64)
    k, v, q = randn(1, 2, 2, 64), randn(2, 2, 2, 64), randn(3, 2, 4, 64)
    off, tab, mb, lens, n = c.args()

    def call(layer=0, n_seq=1, rope=None, mb=mb, tokens=2, **kw):
        K.kvs_append(c.pool, layer, k, v, tokens, off, tab, mb, lens, n_seq, rope=rope, **kw)

    for kw in (dict(layer=1), dict(layer=-1), dict(mb=0), dict(tokens=-1), dict(q=q, n_q_heads=4), dict(n_q_heads=4),
               dict(q_out=torch.empty_like(q), n_q_heads=4), dict(rope=K.RopeAxes(1e4, (31,))),
               dict(rope=K.RopeAxes(1e4, (16, 16)))):
        with pytest.raises((K.KvsError, ValueError)):
            call(**kw)
    with pytest.raises(ValueError):
        call(n_seq=2)                        # offsets and lengths of one sequence
    with pytest.raises(ValueError):
        K.kvs_append(c.pool, 0, k.float(), v, 2, off, tab, mb, lens, 1)
    with pytest.raises(ValueError):
        K.kvs_append(c.pool, 0, k, v[:, :1], 2, off, tab, mb, lens, 1)
    wide = randn(5, 2, 8, 64)
    with pytest.raises((K.KvsError, ValueError)):
        call(q=wide[:, :4], n_q_heads=4, q_out=wide[:, :4])
    assert K.kvs_pool_check(c.pool) == 0
    call(tokens=0)


def test_rows_of_other_shapes_are_refused():
    ok = torch.zeros(4, 6, 64, dtype=torch.bfloat16, device=DEV)
    assert K._rows(ok[:, 2:4], 4, 2, 64, "x") == (ok.data_ptr() + 2 * 64 * 2, 6 * 64)
    assert K._rows(ok, 3, 6, 64, "x")[1] == 6 * 64
    for bad in (ok[:3], ok[:, :, ::2], ok.transpose(0, 1), ok[0], ok[:, ::2], ok.cpu()):
        with pytest.raises(ValueError):
            K._rows(bad, 4, 6, 64, "x")
    for bad in (torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)[::2],
                torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            K._ints(bad, 4, "tok_off")


def test_append_to_a_far_block():
    """Rows behind 2^31 bytes of a slab (and past 2^30 elements)."""
    hkv, d, cap = 32, 128, 18000                   # 18,000 blocks of 131,072 bytes
    k, v = (torch.zeros(cap, hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pool = K.kvs_pool_create(1, hkv, d, 16, K.KVS_DTYPE_BF16, cap, 1, [k], [v])
    kn, vn = randn(1, 20, hkv, d), randn(2, 20, hkv, d)
    table, lens, off = H.i32([[cap - 1, cap - 2]]), H.i32([20]), H.i32([0, 20])
    K.kvs_append(pool, 0, kn, vn, 20, off, table, 2, lens, 1)
    assert torch.equal(k[cap - 1], kn[:16].transpose(0, 1)) and torch.equal(v[cap - 2, :, :4], vn[16:].transpose(0, 1))
    assert not k[: cap - 2].any() and not v[: cap - 2].any() and not k[cap - 2, :, 4:].any()
    q, out = randn(3, 20, hkv, d), torch.empty(20, hkv, d, dtype=torch.bfloat16, device=DEV)
    ws = H.workspace(K.kvs_extend_workspace_size(pool, 20, 1, 2, hkv))
    K.kvs_extend_attn(pool, 0, q, 20, off, hkv, table, 2, lens, 1, True, d ** -0.5, out, ws)
    assert K.kvs_pool_check(pool) == 0
    assert torch.equal(out[0], vn[0])              # the first row sees itself alone


def test_append_in_a_graph_and_on_another_stream():
    c = Case([1, 1, 1], [5, 40, 16], 2, 128)
    k, v = randn(1, 3, 2, 128), randn(2, 3, 2, 128)
    ax = K.RopeAxes(1e6, (64,))
    off, tab, mb, lens, n = c.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        K.kvs_append(c.pool, 0, k, v, 3, off, tab, mb, lens, n, rope=ax)
    k.copy_(randn(7, 3, 2, 128))
    lens += 1                               # the next token of each
    graph.replay()
    torch.cuda.synchronize()
    a = [s.clone() for s in c.slabs]
    with torch.cuda.stream(side):
        K.kvs_append(c.pool, 0, k, v, 3, off, tab, mb, lens, n, rope=ax)
    side.synchronize()
    assert torch.equal(a[0], c.slabs[0]) and torch.equal(a[1], c.slabs[1])
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    K.kvs_gather(c.pool, 0, 3, off, tab, mb, lens, n, k2, v2)
    assert_rotated(f64(k2), OE.rotate_axes(f64(k), lens.cpu().numpy()[None] - 1, 1e6, (64,)))


def test_gather_feeds_the_selection():
    """The cached keys of a span, read back, against refreshed ones."""
    hkv, d = 8, 128
    c = Case([300, 64], [10, 0], hkv, d)
    k, v = randn(1, c.tokens, hkv, d), randn(2, c.tokens, hkv, d)
    c.append(k, v)
    kc, vc = torch.empty_like(k), torch.empty_like(v)
    c.gather(kc, vc)
    kn = kc.clone()
    kn[[5, 17, 250, 310]] += 1
    off = H.i64(c.off)
    idx = torch.full((c.tokens,), -1, dtype=torch.int32, device=DEV)
    idx_off = torch.zeros(3, dtype=torch.int64, device=DEV)
    ws = H.workspace(4 * 2 * 300)
    K.kvs_select_critical(kc, kn, off, 2, 300, hkv * d, 0.01, idx, idx_off, ws)
    got = idx.cpu().numpy()[: int(idx_off[2])]
    assert got.tolist() == [5, 17, 250, 10]
