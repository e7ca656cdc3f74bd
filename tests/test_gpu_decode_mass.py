"""Decode attention with the tokens' weights, over bf16 and microscaled pools, against the fp64 oracle.

Tolerances.  A score is a sum of d products in float32, at worst d roundings of 2^-23 (a tensor core's sum may cut) of
sum |q k| scale, and its exponent's argument two more: a weight before normalisation is off by delta = (d + 4) 2^-23 big
+ 2^-21 (the exponential), relative.  Sums over L tokens, 16 or 32 to a product, add (L / 16 + 64) 2^-23; a weight that
multiplies values keeps 16 bits (2 * 2^-9 * 2^-9 = 2^-17).  Numerator and denominator count once each.  Over microscaled pools the two parts of a weight
are fp16, whose smallest step is 2^-24; weights stand at 2^11 times their share of the reference (which the sum is not
below), so a weight may lose 2^-25 / 2^11 = 2^-36, of the sum, of the largest value: it matters for channels in which the
heavy tokens hold zeros."""
import numpy as np
import pytest
import torch

from oracle import mass as OM
from oracle import mx4 as O4
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace

pytestmark = pytest.mark.gpu

BLOCK = {"bf16": 16, "mx4": 64}


def f64(t):
    return t.double().cpu().numpy()


def make(kind, lens, hq, hkv, d, seed=0, scales=(119, 129), mb_extra=1, layers=1):
    """A pool of shuffled blocks, what lies behind a sequence's end (and in unused blocks) NaN."""
    r, g = np.random.default_rng(seed), torch.Generator(device=DEV).manual_seed(seed)
    block = BLOCK[kind]
    nb = [-(-max(0, x) // block) for x in lens]
    mb, cap = max(max(nb), 1) + mb_extra, sum(nb) + 2
    ids, table, at = r.permutation(cap), np.full((len(lens), mb), -1), 0
    for a, n in enumerate(nb):
        table[a, :n] = ids[at:at + n]
        at += n
    behind = torch.ones(cap, block, dtype=torch.bool, device=DEV)
    for a, n in enumerate(lens):
        for b in range(nb[a]):
            behind[table[a, b], : n - b * block] = False
    s = dict(kind=kind, table=table, mb=mb, cap=cap, block=block, hq=hq, hkv=hkv, d=d, lens=list(lens))
    if kind == "bf16":
        kv = []
        for _ in range(2 * layers):
            x = torch.randn(cap, hkv, block, d, generator=g, device=DEV).to(torch.bfloat16)
            x.transpose(1, 2)[behind] = float("nan")
            kv.append(x)
        s.update(k=kv[:layers], v=kv[layers:], values=[np.nan_to_num(f64(x)) for x in kv])
        s["pool"] = K.kvs_pool_create(layers, hkv, d, block, K.KVS_DTYPE_BF16, cap, len(lens), s["k"], s["v"])
    else:
        codes = [torch.randint(0, 256, (cap, hkv, block, d // 2), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2 * layers)]
        sc = [torch.randint(*scales, (cap, hkv, block, d // 32), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2 * layers)]
        s["values"] = [np.where(behind.cpu().numpy()[:, None, :, None], 0.0, O4.dequantize(c.cpu().numpy(), e.cpu().numpy()))
                       for c, e in zip(codes, sc)]
        for e in sc:
            e.transpose(1, 2)[behind] = 255
        s.update(k=codes[:layers], v=codes[layers:], ksc=sc[:layers], vsc=sc[layers:])
        s["pool"] = K.kvs_pool_create(layers, hkv, d, block, K.KVS_DTYPE_MX4, cap, len(lens), s["k"], s["v"], s["ksc"], s["vsc"])
    s["q"] = (1.5 * torch.randn(len(lens), hq, d, generator=g, device=DEV)).to(torch.bfloat16)
    s["mass_in"] = torch.rand(len(lens), mb * block, generator=g, device=DEV) * hq / max(1, np.mean(np.maximum(lens, 0)))
    s["scale"] = d ** -0.5 if kind == "bf16" else d ** -0.5 / 4
    return s


def call(s, carry=0.75, mass_in="given", layer=0, ws=None, out=None, mass=None, q=None, stream=None):
    n = len(s["lens"])
    out = torch.full((n, s["hq"], s["d"]), float("nan"), device=DEV) if out is None else out
    mass = torch.full_like(s["mass_in"], -3.0) if mass is None else mass
    m_in = s["mass_in"] if isinstance(mass_in, str) else mass_in
    ws = workspace(K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MASS, n, s["mb"], s["hq"])).fill_(0xC3) if ws is None else ws
    a = (s["pool"], layer, s["q"] if q is None else q, s["hq"], i32(s["table"]), s["mb"], i32(s["lens"]), n, s["scale"], out)
    if s["kind"] == "bf16":
        K.kvs_decode_attn_mass(*a, m_in, carry, mass, ws, stream=stream)
    else:
        K.kvs_decode_attn_mx4(*a, ws, mass_in=m_in, carry=carry, mass=mass, stream=stream)
    return out, mass


def check(s, out, mass, carry=0.75, mass_in="given", lens=None, layer=0, before=-3.0, flags=0):
    assert K.kvs_pool_check(s["pool"]) == flags
    n, L = len(s["lens"]), s["mb"] * s["block"]
    lens = s["lens"] if lens is None else lens
    layers = len(s["k"])
    want, mag, w, big = OM.attend(f64(s["q"]), s["values"][layer], s["values"][layers + layer], s["table"], range(n + 1), lens,
                                  s["block"], s["scale"], False)
    delta = (s["d"] + 4) * 2.0 ** -23 * big + 2.0 ** -21
    rel = 2 * (delta + (max(lens + [1]) / 16 + 64) * 2.0 ** -23)
    err = np.abs(f64(out) - want)
    floor = max(lens + [1]) * 2.0 ** -36 * np.abs(s["values"][layers + layer]).max() if s["kind"] == "mx4" else 0.0
    assert (err <= mag * (rel + 2.0 ** -17) + floor + 1e-30).all(), (s["kind"], (err / np.maximum(mag, 1e-30)).max())
    got = f64(mass)
    m_in = np.zeros((n, L)) if mass_in is None else f64(s["mass_in"])
    for a in range(n):
        x = lens[a]
        exp = carry * m_in[a, :x] + w[a]
        assert (np.abs(got[a, :x] - exp) <= w[a] * (rel + s["hq"] * 2.0 ** -24) + 2.0 ** -23 * exp + 1e-37).all()
        assert (got[a, x:] == before).all()
    return np.linalg.norm(f64(out) - want) / max(np.linalg.norm(want), 1e-30)


SHAPES = [   # heads and channels
    ("bf16", 8, 8, 64), ("bf16", 8, 2, 64), ("bf16", 8, 1, 64), ("bf16", 12, 1, 64), ("bf16", 32, 2, 64),
    ("bf16", 4, 4, 128), ("bf16", 6, 2, 128), ("bf16", 16, 2, 128), ("bf16", 20, 4, 128), ("bf16", 12, 1, 128), ("bf16", 16, 1, 128),
    ("bf16", 9, 1, 128), ("mx4", 4, 4, 128), ("mx4", 8, 2, 128), ("mx4", 8, 1, 128), ("mx4", 7, 1, 128), ("mx4", 12, 1, 128),
    ("mx4", 32, 2, 128),
]


@pytest.mark.parametrize("kind, hq, hkv, d", SHAPES)
@pytest.mark.parametrize("lens", [[1], [0, 1, 15, 16, 17, 31, 33, 64, 65], [300, 384, 0, 321], [5000, 1, 2047]])
def test_decode_mass(kind, hq, hkv, d, lens):
    s = make(kind, lens, hq, hkv, d, seed=len(lens) + hq)
    rel = check(s, *call(s))
    assert rel <= 2e-5


@pytest.mark.parametrize("kind, hq, hkv", [("bf16", 2, 1), ("mx4", 8, 1)])
def test_one_long_sequence_over_all_ctas(kind, hq, hkv):
    s = make(kind, [40000], hq, hkv, 128)
    check(s, *call(s))


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_many_short_sequences(kind):
    lens = np.random.default_rng(3).integers(0, 40, 700).tolist()
    s = make(kind, lens, 4, 2, 128)
    check(s, *call(s))


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("n, most", [(31, 900), (32, 300), (33, 700), (63, 200), (64, 1500), (65, 400)])
def test_sequences_around_what_a_warp_places(kind, n, most):
    lens = np.random.default_rng(n).integers(0, most, n)
    lens[[0, n // 2, n - 1]] = 0, 1, most
    s = make(kind, lens.tolist(), 8, 2, 128 if kind == "mx4" else 64, seed=n)
    check(s, *call(s))


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_mass_forms(kind):
    """No earlier masses, in place, carried whole; no masses at all (microscaled); twice the same to the bit."""
    s = make(kind, [700, 33], 8, 2, 128)
    out, mass = call(s, mass_in=None, carry=5.0)
    check(s, out, mass, mass_in=None)
    own = s["mass_in"].clone()
    out2, own = call(s, mass_in=own, carry=1.0, mass=own)
    assert torch.equal(out, out2)
    for a, n in enumerate(s["lens"]):
        assert torch.equal(own[a, n:], s["mass_in"][a, n:])
        torch.testing.assert_close(own[a, :n], s["mass_in"][a, :n] + mass[a, :n], rtol=2.0 ** -22, atol=1e-38)
    out3, mass3 = call(s, mass_in=None)
    assert torch.equal(out, out3) and torch.equal(mass, mass3)
    if kind == "mx4":
        n, o = len(s["lens"]), torch.empty_like(out)
        ws = workspace(K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MASS, n, s["mb"], 8))
        K.kvs_decode_attn_mx4(s["pool"], 0, s["q"], 8, i32(s["table"]), s["mb"], i32(s["lens"]), n, s["scale"], o, ws)
        assert torch.equal(o, out)


def test_microscaled_scales_of_every_size():
    """Scales over 40 binary orders: values far below a group's largest, and queries far from 1."""
    for seed, (lo, hi) in enumerate([(1, 40), (100, 141), (200, 230)]):
        s = make("mx4", [200, 64, 515], 8, 2, 128, seed=seed, scales=(lo, hi))
        s["scale"] = 0.05 * 2.0 ** (127 - hi + 1)
        # values are compared to the largest of their 32 channels in the sequence: 2^-27 of it is lost
        check(s, *call(s))


def test_microscaled_smallest_scales():
    """Byte 0 is 2^-127, not 0: keys of that size count where the scale brings them up."""
    s = make("mx4", [200, 64, 515], 8, 2, 128, seed=5, scales=(0, 3))
    s["scale"] = 0.05 * 2.0 ** 125
    out, mass = call(s)
    check(s, out, mass)
    zero = [x.clone() for x in s["ksc"]]
    for x in s["ksc"]:
        x[x < 255] = 0
    s["values"][0] = s["values"][0] * np.repeat(np.exp2(-np.where(zero[0].cpu().numpy() < 255, zero[0].cpu().numpy(), 0).astype(np.float64)), 32, -1)
    check(s, *call(s))


def test_workspaces_for_a_step_serve_smaller_ones():
    s = make("mx4", [64], 8, 2, 128)
    many = K.kvs_pool_create(1, 2, 128, 64, K.KVS_DTYPE_MX4, s["cap"], 4096, s["k"], s["v"], s["ksc"], s["vsc"])
    for op in (K.KVS_OP_DECODE_MASS, K.KVS_OP_COMPACT):
        size = np.array([[K.kvs_workspace_size(many, op, n, b, 8) for b in (1, 2, 30, 500, 4096)] for n in (1, 2, 33, 600, 4096)])
        assert (np.diff(size, axis=0) >= 0).all() and (np.diff(size, axis=1) >= 0).all()


def test_scores_far_apart():
    """A maximum that keeps moving, and weights below every other's rounding."""
    for kind in ("bf16", "mx4"):
        s = make(kind, [900, 130], 8, 2, 128, seed=7)
        s["scale"] *= 8
        check(s, *call(s))


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
def test_bad_blocks_and_lengths(kind):
    s = make(kind, [300, 200, 64], 8, 2, 128)
    s["table"][0, 1], s["table"][1, :], s["table"][2, 0] = s["cap"], -5, s["table"][2, 0]
    check(s, *call(s), flags=K.KVS_DEVERR_BLOCK_ID)
    s = make(kind, [90, 3], 8, 2, 128, mb_extra=0)
    s["lens"] = [s["mb"] * s["block"] + 1, -4]
    s["values"] = [np.nan_to_num(x) for x in s["values"]]
    out, mass = call(s)
    assert K.kvs_pool_check(s["pool"]) == K.KVS_DEVERR_SEQ_LEN
    assert (out[1] == 0).all() and (mass[1] == -3).all()


def test_layers_streams_and_graphs():
    """Layers added up in place on another stream, captured and replayed with new queries."""
    s = make("bf16", [400, 1000, 77], 16, 2, 128, layers=3)
    n, mb = 3, s["mb"]
    table, lens = i32(s["table"]), i32(s["lens"])
    ws = workspace(K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MASS, n, mb, 16))
    q, out, mass = s["q"].clone(), [torch.empty(n, 16, 128, device=DEV) for _ in range(3)], torch.zeros_like(s["mass_in"])
    side = torch.cuda.Stream()

    def step():
        mass.zero_()
        for l in range(3):
            K.kvs_decode_attn_mass(s["pool"], l, q, 16, table, mb, lens, n, s["scale"], out[l], mass, 1.0, mass, ws)
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        q.copy_(-s["q"])
        s["q"] = q
        graph.replay()
        side.synchronize()
    total = torch.zeros_like(mass)
    for l in range(3):
        o, m = call(s, layer=l, mass_in=None)
        check(s, o, m, layer=l, mass_in=None)
        assert torch.equal(o, out[l])
        total += m.clamp(min=0)
    torch.testing.assert_close(mass, total, rtol=1e-6, atol=0)


def test_refusals():
    s = make("bf16", [40], 8, 2, 64)
    mx = make("mx4", [40], 8, 2, 128)
    n, mb, table, lens, pool = 1, s["mb"], i32(s["table"]), i32(s["lens"]), s["pool"]
    out, mass = torch.empty(1, 8, 64, device=DEV), torch.zeros_like(s["mass_in"])
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_DECODE_MASS, n, mb, 8))
    good = dict(pool=pool, layer=0, q=s["q"], n_q_heads=8, block_table=table, max_blocks=mb, seq_len=lens, n_seq=1, scale=0.1,
                out=out, mass_in=s["mass_in"], carry=1.0, mass=mass, ws=ws)
    K.kvs_decode_attn_mass(**good)
    bad = [dict(pool=mx["pool"], q=mx["q"], out=torch.empty(1, 8, 128, device=DEV), mass_in=None,
                mass=torch.zeros_like(mx["mass_in"]), block_table=i32(mx["table"]), max_blocks=mx["mb"]),
           dict(layer=1), dict(layer=-1), dict(n_q_heads=7, q=s["q"][:, :7].contiguous()), dict(scale=0.0), dict(scale=float("nan")),
           dict(scale=3e38), dict(carry=float("inf")), dict(max_blocks=mb - 1), dict(ws=ws[:16]), dict(ws=ws.cpu()),
           dict(mass=mass[:, :-1]), dict(mass=mass.double()), dict(mass=None), dict(out=out.to(torch.bfloat16)), dict(q=s["q"].float()),
           dict(q=s["q"].cpu()), dict(seq_len=lens.long()), dict(n_seq=2)]
    for change in bad:
        with pytest.raises((K.KvsError, ValueError)):
            K.kvs_decode_attn_mass(**{**good, **change})
    with pytest.raises(K.KvsError):
        K.kvs_decode_attn_mx4(pool, 0, s["q"], 8, table, mb, lens, 1, 0.1, out, ws)
    K.kvs_decode_attn_mass(**{**good, "n_seq": 0})
    assert K.kvs_pool_check(pool) == 0
