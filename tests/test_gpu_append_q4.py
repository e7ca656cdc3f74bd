"""The append into 4-bit pools and the way back: head counts that mix keys,
values and queries in a warp, given positions, groups made for the quantiser's
decisions, and every value read back."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from oracle import extend as OE
import harness as H
from test_gpu_append import SECTIONS, Case, assert_rotated, f64, randn

DEV = H.DEV


def quantised(k, v):
    """kvs_quantize_q4 of rows [n][hkv][128]: (codes K, codes V, scales K,
    scales V), each [n][hkv][...], on the host."""
    n, hkv, d = k.shape
    nb = -(-n // 256)
    blocks = lambda x: torch.cat([x, torch.zeros(nb * 256 - n, hkv, d, dtype=x.dtype, device=DEV)]).view(nb, 256, hkv, d).transpose(1, 2).contiguous()  # noqa: E731,E501
    s = [torch.zeros(nb, hkv, 256, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
        [torch.zeros(nb, hkv, 256, 2, 2, dtype=torch.float16, device=DEV) for _ in range(2)]
    p = K.kvs_pool_create(1, hkv, d, 256, K.KVS_DTYPE_Q4G64, nb, 1, [s[0]], [s[1]], [s[2]], [s[3]])
    K.kvs_quantize_q4(p, 0, blocks(k), blocks(v), H.i32(np.arange(nb)), nb)
    assert K.kvs_pool_check(p) == 0
    return [t.transpose(1, 2).reshape(nb * 256, hkv, *t.shape[3:])[:n].cpu().numpy() for t in s]


def values(code, sb):
    """scale * code + bias in 64 bits, [n][hkv][128]."""
    c = np.stack([code & 15, code >> 4], -1).reshape(*code.shape[:2], 2, 64).astype(np.float64)
    sb = sb.astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (c * sb[..., 0:1] + sb[..., 1:2]).reshape(*code.shape[:2], 128)


def same_bits(a, b):
    np.testing.assert_array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


@pytest.mark.parametrize("new, ctx", [([1] * 5, [0, 255, 256, 700, 31]), ([257, 0, 33], [0, 5, 255]), ([150, 260], [3, 100])])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("hq", [0, 5, 32])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_append_q4_with_queries(new, ctx, hkv, hq, axes):
    """Keys, values and queries of any head count: what a bf16 pool would hold,
    quantised bit for bit; queries rotated; nothing else written; both tensors
    read back."""
    d = 128
    c, b = Case(new, ctx, hkv, d, q4=True, pad=2, seed=hkv), Case(new, ctx, hkv, d, pad=2)
    k, v = randn(31, c.tokens, hkv, d), randn(32, c.tokens, hkv, d)
    q = randn(33, c.tokens, hq, d) if hq else None
    q_out = torch.full_like(q, 5.0) if hq else None
    pl = c.places()
    rows = sorted(pl)
    pos = np.zeros((max(axes, 1), c.tokens), np.int64)
    for t, (_, p, _, _) in pl.items():
        pos[:, t] = p
    kw = {}
    if axes == 3:
        pos = np.random.default_rng(3).integers(0, 70000, (3, c.tokens))
        kw["pos"] = H.i32(pos)
    rope = K.RopeAxes(1e6, SECTIONS[d, axes]) if axes else None
    before = [s.cpu().numpy() for s in c.slabs]
    c.append(k, v, rope=rope, q=q, n_q_heads=hq, q_out=q_out, **kw)
    b.append(k, v, rope=rope, **kw)
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    b.gather(kb, vb)
    assert K.kvs_pool_check(c.pool) == 0 and K.kvs_pool_check(b.pool) == 0
    blk, at = np.array([pl[t][2] for t in rows]), np.array([pl[t][3] for t in rows])
    made = quantised(kb[rows], vb[rows])
    for i in range(4):
        before[i][blk, :, at] = made[i]
        same_bits(c.slabs[i].cpu().numpy(), before[i])
    if hq:
        exp = OE.rotate_axes(f64(q), pos, 1e6, SECTIONS[d, axes]) if axes else f64(q)
        assert_rotated(f64(q_out)[rows], exp[rows])
        assert (q_out[c.tokens - 2:] == 5).all()
    k2, v2 = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    c.gather(k2, v2)
    for got, code, sb in ((k2, made[0], made[2]), (v2, made[1], made[3])):
        val = values(code, sb)
        # one rounding to bf16 (half a step: 2^-8 relative) of a float32 sum (2^-24)
        assert (np.abs(f64(got)[rows] - val) <= 2.0 ** -8 * (1 + 2.0 ** -15) * np.abs(val) + 1e-30).all()
        assert (got[c.tokens - 2:] == 3).all()
    assert K.kvs_pool_check(c.pool) == 0


def special_groups():
    """Groups of 64 bf16 values whose codes are decided at a border."""
    r = np.random.default_rng(0)
    out = []
    for step in (1.0, 2.0, 2.0 ** -9, 2.0 ** 9):            # 15 steps from the least to the largest value
        for base in (0.0, -7.5, 1.0, -15.0):
            half = (r.integers(0, 15, 64) + 0.5) * step     # quotients of exactly a half: to the even code
            half[0], half[1] = 0.0, 15 * step
            out.append(half + base * step)
            near = half * (1 + r.choice([-1, 1], 64) * 2.0 ** -8)     # one bf16 step off a half
            near[0], near[1] = 0.0, 15 * step
            out.append(near)
    for s in (0.1, 0.3, 1.7, 77.0, 1e-3):                   # steps that are no power of two
        x = (r.integers(0, 15, 64) + 0.5) * s
        x[0], x[1] = 0.0, 15 * s
        out.append(x - 4 * s)
    for x in (0.0, -0.0, 0.5, -3.0, 1e-40, 7e4, -1e38):     # constant groups
        out.append(np.full(64, x))
    mixed = np.zeros(64)
    mixed[::2] = -0.0
    out.append(mixed)
    out.append(-mixed)
    out.append(r.normal(0, 1e-38, 64))                      # subnormal, and scales that vanish in fp16
    out.append(r.normal(0, 1e-6, 64))
    out.append(r.normal(0, 1e5, 64))                        # biases outside fp16
    out.append(r.normal(0, 1e6, 64))                        # scales outside fp16
    out.append(r.normal(0, 1e30, 64))
    out.append(np.where(r.random(64) < 0.5, 3.3e38, -3.3e38))   # a range outside float32
    for odd in ([np.inf], [-np.inf], [np.inf, -np.inf], [np.nan], [np.nan, np.inf], [np.nan, -np.inf, np.inf]):
        x = r.normal(0, 1, 64)
        x[r.choice(64, len(odd), replace=False)] = odd
        out.append(x)
    out.append(np.full(64, np.inf))
    out.append(np.full(64, -np.inf))
    return np.array(out)


def test_groups_at_the_quantisers_borders():
    """Halves, one step off them, constants, signed zeros, subnormals, values
    and ranges that fp16 or float32 does not hold, infinities and NaN: bit for
    bit what kvs_quantize_q4 stores, in every place of a row."""
    g = special_groups()
    hkv, d = 2, 128
    n = -(-len(g) // 2)
    for shift in range(4):                  # each group in the keys and values, in both halves of a row
        rows = np.resize(np.roll(g, shift, 0), (2 * n, 64)).reshape(n, 1, d)
        k = torch.from_numpy(np.concatenate([rows, np.roll(rows, 3, 0)], 1)).float().to(DEV).to(torch.bfloat16)
        v = k.flip(0).contiguous()
        c = Case([n], [250], hkv, d, q4=True)
        c.append(k, v)
        assert K.kvs_pool_check(c.pool) == 0
        pl = c.places()
        blk, at = np.array([pl[t][2] for t in range(n)]), np.array([pl[t][3] for t in range(n)])
        made = quantised(k, v)
        for i in range(4):
            same_bits(c.slabs[i].cpu().numpy()[blk, :, at], made[i])


def test_quotients_near_a_half():
    """Random bf16 groups by the hundred thousand: among them quotients within
    1e-4 of a half, where the product with the reciprocal does not decide."""
    n, hkv, d = 4096, 8, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.rand(n, hkv, d, generator=g, device=DEV)
    k, v = (x * 3 - 1).to(torch.bfloat16), torch.randint(-60, 61, (n, hkv, d), generator=g, device=DEV).to(torch.bfloat16)
    made = quantised(k, v)
    # the inputs do reach the case
    sb = made[3].astype(np.float64)
    quo = (f64(v).reshape(n, hkv, 2, 64) - sb[..., 1:2]) / sb[..., 0:1]
    assert (np.abs(quo - np.floor(quo) - 0.5) < 1e-4).sum() > 1000
    c = Case([n], [0], hkv, d, q4=True)
    c.append(k, v)
    pl = c.places()
    blk, at = np.array([pl[t][2] for t in range(n)]), np.array([pl[t][3] for t in range(n)])
    for i in range(4):
        same_bits(c.slabs[i].cpu().numpy()[blk, :, at], made[i])
