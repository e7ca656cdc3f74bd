"""A pool of microscaled 4-bit values: append, read-back, block copies, export, compaction."""
import numpy as np
import pytest
import torch

from oracle import extend as OE
from oracle import mx4 as O4
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace
from test_gpu_compact import make_pool, run_compact

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def append(k, v, lens, new, hkv, rope=None, pos=None, q=None, q_out=None, pad=0):
    """One append into a fresh pool whose bytes are 0x5A, and its read-back."""
    block, n, T = 64, len(lens), k.shape[0]
    nb = [-(-x // block) for x in lens]
    mb, cap = max(max(nb), 1), sum(nb) + 1
    ids, table, at = np.random.default_rng(T).permutation(cap), np.full((n, mb), -1), 0
    for a, x in enumerate(nb):
        table[a, :x] = ids[at:at + x]
        at += x
    full = lambda w: torch.full((cap, hkv, block, w), 0x5A, dtype=torch.uint8, device=DEV)  # noqa: E731
    kc, vc, ks, vs = full(64), full(64), full(4), full(4)
    pool = K.kvs_pool_create(1, hkv, 128, block, K.KVS_DTYPE_MX4, cap, n, [kc], [vc], [ks], [vs])
    off = np.concatenate([[0], np.cumsum(new)]) + pad
    args = (i32(off), i32(table), mb, i32(lens), n)
    K.kvs_append(pool, 0, k, v, T, *args, pos=pos, rope=rope, q=q, n_q_heads=0 if q is None else q.shape[1], q_out=q_out)
    kb, vb = torch.full((T, hkv, 128), -5.0, dtype=torch.bfloat16, device=DEV), torch.full((T, hkv, 128), -5.0, dtype=torch.bfloat16, device=DEV)
    K.kvs_gather(pool, 0, T, *args, kb, vb)
    assert K.kvs_pool_check(pool) == 0
    return dict(kc=kc, vc=vc, ks=ks, vs=vs, table=table, off=off, kb=kb, vb=vb, where=OE.places(off, lens, table, block))


def held(x):
    c, s = O4.quantize(x)
    return c, s, O4.dequantize(c, s)


@pytest.mark.parametrize("lens, new, hkv", [([1], [1], 1), ([70, 64, 9], [7, 64, 9], 2), ([200, 0, 5, 65], [130, 0, 2, 1], 3),
                                            ([2000, 300], [700, 300], 8)])
@pytest.mark.parametrize("size", [0, -100, 100])
def test_append_is_the_oracles_to_the_bit(lens, new, hkv, size):
    g = torch.Generator(device=DEV).manual_seed(sum(new))
    T, pad = sum(new), 3
    x = [torch.ldexp(torch.randn(T + 2 * pad, hkv, 128, generator=g, device=DEV), torch.tensor(size, device=DEV)).to(torch.bfloat16) for _ in range(2)]
    for t in x:   # zeros, equal values, ties, and groups of very different size
        t[:, 0, :32] = 0
        t[::2, :, 32:64] = t[::2, :, 32:33]
        t[1::3, :, 64:96] = torch.round(t[1::3, :, 64:96].float() * 4).to(torch.bfloat16) / 4
        t[:, :, 96:] *= 1024
    r = append(x[0], x[1], lens, new, hkv, pad=pad)
    touched = np.zeros((r["kc"].shape[0], 64), bool)
    for t, (_, _, phys, at) in r["where"].items():
        touched[phys, at] = True
        for src, code, scale, back in ((x[0], "kc", "ks", "kb"), (x[1], "vc", "vs", "vb")):
            c, s, y = held(f64(src[t]))
            np.testing.assert_array_equal(r[code][phys, :, at].cpu().numpy(), c)
            np.testing.assert_array_equal(r[scale][phys, :, at].cpu().numpy(), s)
            np.testing.assert_array_equal(f64(r[back][t]), y)
    for name in ("kc", "vc", "ks", "vs"):     # every other row is as it was
        assert (r[name].transpose(1, 2)[torch.as_tensor(~touched, device=DEV)] == 0x5A).all()
    rest = torch.ones(T + 2 * pad, dtype=torch.bool, device=DEV)
    rest[list(r["where"])] = False
    assert (r["kb"][rest] == -5).all() and (r["vb"][rest] == -5).all()


def test_extremes_of_bf16():
    """Subnormals, the largest finite values, infinities (held as the largest code) and a NaN beside whole groups."""
    x = torch.zeros(4, 1, 128)
    x[0, 0, :32] = 2.0 ** -130
    x[0, 0, 32:64] = torch.linspace(-1, 1, 32) * 3.3e38
    x[1, 0, 0], x[1, 0, 1] = float("inf"), -3.0e38
    x[1, 0, 64:] = 1.0
    x[2, 0, :32] = 2.0 ** -126
    x[3, 0, 5] = float("nan")
    x[3, 0, 32:] = 7.0
    xb = x.to(torch.bfloat16).to(DEV)
    r = append(xb, xb, [4], [4], 1)
    got = f64(r["kb"])
    assert np.isfinite(got).all()
    for t, sl in ((0, slice(0, 128)), (1, slice(32, 128)), (2, slice(0, 128)), (3, slice(32, 128))):
        np.testing.assert_array_equal(got[t, 0, sl], held(f64(xb[t]))[2][0, sl])
    # the largest finite exponent is 127, so the group's scale is 2^125, and 6 and -6 of it are the ends
    assert got[1, 0, 0] == 6 * 2.0 ** 125 and got[1, 0, 1] == -6 * 2.0 ** 125


def test_rotated_append_with_queries():
    """Keys are rotated in float32, rounded to bf16 and quantised: codes may differ from the oracle's where the rotated
    value lies on a border of bf16 or of a code, and then by one step; queries as in a bf16 pool."""
    g = torch.Generator(device=DEV).manual_seed(4)
    lens, new, hkv, hq = [900, 70], [300, 70], 2, 8
    T = sum(new)
    k, v = (torch.randn(T, hkv, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, hq, 128, generator=g, device=DEV).to(torch.bfloat16)
    q_out = torch.empty_like(q)
    r = append(k, v, lens, new, hkv, rope=K.RopeAxes(1e6, (64,)), q=q, q_out=q_out)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])[None]
    want = OE.rotate_axes(f64(k), pos, 1e6, (64,))
    rounded = f64(torch.as_tensor(want).to(torch.bfloat16))
    y = held(rounded)[2]
    got = f64(r["kb"])
    assert (got != y).mean() < 1e-3
    step = np.exp2(np.floor(np.log2(np.abs(rounded.reshape(T, hkv, 4, 32)).max(-1, keepdims=True)))).repeat(32, -1).reshape(y.shape)
    assert (np.abs(got - y) <= step).all()      # 2 scales: the widest step of a code, or a scale one power apart
    np.testing.assert_array_equal(f64(r["vb"]), held(f64(v))[2])
    rq = OE.rotate_axes(f64(q), pos, 1e6, (64,))
    assert (np.abs(f64(q_out) - rq) <= 2.0 ** -8 * np.abs(rq) + 1e-5).all()


@pytest.mark.parametrize("lens, part, shared", [([300, 64, 1], 0.5, [0, 0, 0]), ([3000, 2900], 0.3, [0, 40]), ([70000], 0.6, [0])])
def test_compact(lens, part, shared):
    run_compact("mx4", 2 if len(lens) > 1 else 1, 2 if len(lens) > 1 else 1, 128, lens, part, shared, True, cap_extra=60)


def test_copy_on_write_export_import_and_stats():
    pool, slabs, block = make_pool("mx4", 2, 2, 128, 6, 3)
    bytes_ = K.kvs_pool_block_bytes(pool)
    assert bytes_ == 2 * 2 * 2 * 64 * 68
    table, refs = i32([[0, 1], [0, 2], [3, -1]]), i32([2, 1, 1, 1, 0, 0])
    free, n_free = i32([5, 4, 0, 0, 0, 0]), i32([2])
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_BLOCKS, 3, 2))
    before = [s.clone() for s in slabs]
    K.kvs_block_write(pool, table, 2, 3, i32([1]), i32([0]), 1, refs, free, n_free, ws)
    assert table.tolist() == [[0, 1], [4, 2], [3, -1]]
    for s, x in zip(slabs, before):
        assert torch.equal(s[4], x[0]) and torch.equal(s[:4], x[:4])
    packed = torch.empty(2 * bytes_, dtype=torch.uint8, device=DEV)
    K.kvs_pool_export(pool, i32([2, 3]), 2, packed)
    K.kvs_pool_import(pool, i32([5, 1]), 2, packed)
    for s, x in zip(slabs, before):
        assert torch.equal(s[5], x[2]) and torch.equal(s[1], x[3])
    stats = K.kvs_pool_stats(pool, refs, i32([4]))
    assert stats["unique_blocks"] == 4 and stats["pool_bytes"] == 4 * bytes_
    assert K.kvs_pool_check(pool) == 0


def test_pool_refusals():
    x = lambda *s: [torch.zeros(*s, dtype=torch.uint8, device=DEV)]  # noqa: E731
    k, sc, dt = x(4, 2, 64, 64), x(4, 2, 64, 4), K.KVS_DTYPE_MX4
    K.kvs_pool_create(1, 2, 128, 64, dt, 4, 2, k, k, sc, sc)
    d = x(2, 2, 16, 256)
    for args, more in (((1, 2, 64, 64, dt, 4, 2, k, k, sc, sc), {}), ((1, 2, 128, 16, dt, 4, 2, k, k, sc, sc), {}),
                       ((1, 2, 128, 64, dt, 4, 2, k, k), {}),
                       ((1, 2, 128, 64, dt, 4, 2, k, k, sc, sc), dict(dk_layers=d, dv_layers=d, diff_capacity_blocks=2))):
        with pytest.raises(K.KvsError):
            K.kvs_pool_create(*args, **more)
    pool = K.kvs_pool_create(1, 2, 128, 64, dt, 4, 2, k, k, sc, sc)
    q, out, ws = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 8, 128, device=DEV), workspace(1 << 20)
    t, n = i32([[0]]), i32([5])
    for refused in (lambda: K.kvs_decode_attn(pool, 0, q, 8, t, 1, n, 1, None, None, None, 1e4, 0.1, out, ws),
                    lambda: K.kvs_decode_attn_q4(pool, 0, q, 8, t, 1, n, 1, 0.1, out, ws),
                    lambda: K.kvs_quantize_q4(pool, 0, q, q, n, 1),
                    lambda: K.kvs_extend_attn(pool, 0, q, 1, i32([0, 1]), 8, t, 1, n, 1, True, 0.1, torch.zeros_like(q), ws)):
        with pytest.raises(K.KvsError):
            refused()
