"""The tokens' weights over query chunks against the fp64 oracle.

Tolerance.  As for decoding (test_gpu_decode_mass): a score is off by at most (d + 4) 2^-23 of sum |q k| scale, the
exponential by 2^-21, relative, in the weight's numerator and in the row's sum; log2 of the sum is rounded to float32
(2^-24 of up to |log2| <= 2 big + 16, times ln 2); sums of n terms add at most 2^-24 of the number of their steps: 128 a
tile, and a tile a step."""
import numpy as np
import pytest
import torch

from oracle import mass as OM
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace
from test_gpu_decode_mass import f64, make

pytestmark = pytest.mark.gpu


def chunk(lens, new, hq, hkv, d, seed=0, pad=0, wide=0):
    s = make("bf16", lens, hq, hkv, d, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    off = np.concatenate([[0], np.cumsum(new)]) + pad
    T = int(off[-1]) + pad
    rows = (1.5 * torch.randn(max(T, 1), hq + wide, d, generator=g, device=DEV)).to(torch.bfloat16)
    q = rows[:, :hq]
    live = torch.zeros(max(T, 1), dtype=torch.bool, device=DEV)
    live[pad:int(off[-1])] = True
    rows[~live] = float("nan")        # rows of no sequence hold anything
    s.update(q=q, off=off, T=T)
    return s


def call(s, causal, carry=0.75, mass_in="given", mass=None, ws=None):
    n = len(s["lens"])
    mass = torch.full_like(s["mass_in"], -3.0) if mass is None else mass
    m_in = s["mass_in"] if isinstance(mass_in, str) else mass_in
    ws = workspace(K.kvs_extend_mass_workspace_size(s["pool"], s["T"], n, s["mb"], s["hq"])).fill_(0xC3) if ws is None else ws
    K.kvs_extend_mass(s["pool"], 0, s["q"], s["T"], i32(s["off"]), s["hq"], i32(s["table"]), s["mb"], i32(s["lens"]), n, causal,
                      s["scale"], m_in, carry, mass, ws)
    return mass


def check(s, mass, causal, carry=0.75, mass_in="given", lens=None, flags=0, before=-3.0):
    assert K.kvs_pool_check(s["pool"]) == flags
    lens = s["lens"] if lens is None else lens
    q = np.nan_to_num(f64(s["q"]))
    _, _, w, big = OM.attend(q, s["values"][0], None, s["table"], s["off"], lens, 16, s["scale"], causal)
    rows = max(int(np.max(np.diff(s["off"]))), 1) * s["hq"]
    rel = 2 * ((s["d"] + 4) * 2.0 ** -23 * big + 2.0 ** -21) + 2.0 ** -24 * (2 * big * 1.45 + 16)
    rel += 2.0 ** -24 * (128 + max(lens + [1]) / 128 + 128 + rows / 128 + s["hkv"] * 16)
    got = f64(mass)
    for a, x in enumerate(lens):
        m = f64(s["mass_in"])[a, :x] * carry if mass_in is not None else 0.0
        assert (np.abs(got[a, :x] - (m + w[a])) <= w[a] * rel + 2.0 ** -23 * (m + w[a]) + 1e-37).all(), a
        assert (got[a, x:] == before).all()


SHAPES = [(8, 8, 64), (8, 2, 64), (12, 1, 64), (16, 1, 64), (4, 4, 128), (6, 2, 128), (16, 2, 128), (20, 4, 128), (9, 1, 128), (7, 1, 128)]
LENS = [   # stored tokens with the new ones, new ones
    ([1], [1]),
    ([5, 40, 16, 129], [5, 1, 0, 128]),
    ([300, 700, 64], [300, 32, 64]),
    ([2500], [17]),
    ([700, 513, 1030], [600, 513, 3]),
]


@pytest.mark.parametrize("hq, hkv, d", SHAPES)
@pytest.mark.parametrize("lens, new", LENS)
@pytest.mark.parametrize("causal", [True, False])
def test_extend_mass(hq, hkv, d, lens, new, causal):
    s = chunk(lens, new, hq, hkv, d, seed=hq + len(lens), pad=2, wide=hq % 3)
    check(s, call(s, causal), causal)


@pytest.mark.parametrize("causal", [True, False])
def test_long_chunks(causal):
    s = chunk([4000, 1500], [3000, 1], 4, 2, 128)
    check(s, call(s, causal), causal)
    s = chunk([9000], [1300], 4, 1, 64)
    check(s, call(s, causal), causal)


def test_key_tiles_that_rows_pass_by():
    """A causal chunk of many row tiles in one piece: the second 128 keys of a pair are seen eight row tiles later."""
    s = chunk([3000], [3000], 64, 8, 64)
    check(s, call(s, True), True)


@pytest.mark.parametrize("lens, new, hq, hkv, d", [
    ([30000, 1, 12000], [32, 0, 5], 16, 8, 64),           # a pair's tiles over more CTAs than the others'
    ([6100, 900, 0, 2000, 129], [4, 1, 0, 3, 4], 32, 32, 64),
    ([5000, 8000, 128], [7, 1, 12], 20, 20, 128),
    ([6100, 900, 0, 2000], [4, 1, 2, 3], 32, 32, 64),     # a row that sees nothing: items instead of stretches
])
@pytest.mark.parametrize("causal", [True, False])
def test_even_stretches(lens, new, hq, hkv, d, causal):
    """Enough key tiles for few rows that every CTA takes an even stretch of them."""
    s = chunk(lens, new, hq, hkv, d, seed=len(lens), pad=1)
    check(s, call(s, causal), causal)


@pytest.mark.parametrize("lens, new, hq, hkv, d", [
    ([300, 40, 7, 0], [20, 1, 1, 0], 16, 2, 128),         # two row tiles beside shorter sequences
    ([1, 16, 128, 129, 127], [1, 16, 3, 2, 1], 8, 8, 64),
    ([900, 10, 1000], [9, 12, 1], 12, 1, 64),             # rows in front of the first key
    ([3900, 4000, 1, 257], [4, 2, 1, 4], 40, 8, 128),     # more tiles than stages, both passes
    ([500] * 30, [4] * 30, 40, 8, 64),                    # more CTAs than SMs
    ([90, 0, 17] * 21 + [128], [1, 0, 2] * 21 + [3], 8, 4, 64),   # 64 sequences
    ([364], [64], 8, 2, 128),                             # more row tiles than sequences
    ([305], [182], 20, 4, 64),
    ([450, 20, 700], [150, 20, 40], 16, 4, 128),
    ([33] * 32 + [700], [1] * 32 + [40], 16, 2, 128),     # 33, the last of several row tiles
    ([33] * 65, [1] * 65, 8, 2, 64),                      # one more than a warp counts
])
@pytest.mark.parametrize("causal", [True, False])
def test_short_calls(lens, new, hq, hkv, d, causal):
    """Few rows and short tables: both passes in one kernel."""
    s = chunk(lens, new, hq, hkv, d, seed=len(lens), pad=1)
    mass = call(s, causal)
    check(s, mass, causal)
    assert torch.equal(call(s, causal), mass)


def test_short_calls_far_scores_bad_blocks_offsets_and_graphs():
    s = chunk([900, 640, 30], [3, 3, 3], 4, 2, 64)
    for b in range(s["k"][0].shape[0]):
        s["k"][0][b] *= 30 if b % 3 == 0 else 0.1 if b % 3 == 1 else 1
    s["values"][0] = np.nan_to_num(f64(s["k"][0]))
    check(s, call(s, True), True)
    ws = workspace(K.kvs_extend_mass_workspace_size(s["pool"], s["T"], 3, s["mb"], 4)).fill_(0xC3)
    off, table, lens, mass, q = i32(s["off"]), i32(s["table"]), i32(s["lens"]), torch.full_like(s["mass_in"], -3.0), s["q"].contiguous()
    run = lambda: K.kvs_extend_mass(s["pool"], 0, q, s["T"], off, 4, table, s["mb"], lens, 3, True, s["scale"], s["mass_in"], 0.75, mass, ws)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        q.neg_()
        for _ in range(3):
            graph.replay()
        side.synchronize()
    s["q"] = q
    check(s, mass, True)
    values = s["values"][0]
    s["table"][0, 1] = -7
    bad = call(s, True)
    assert K.kvs_pool_check(s["pool"]) == K.KVS_DEVERR_BLOCK_ID
    s["table"][0, 1] = s["cap"]
    s["values"][0] = np.concatenate([values, np.zeros((1,) + values.shape[1:])])   # zero keys
    check(s, bad, True)
    s["off"] = np.array([0, 3, 2, 9])
    mass = call(s, True)
    assert K.kvs_pool_check(s["pool"]) & K.KVS_DEVERR_JOB and (mass == -3).all()


def test_scores_out_of_the_reference():
    """The first keys of a row say nothing about the later ones: scores that jump by hundreds, up and down."""
    s = chunk([900, 640], [200, 3], 4, 2, 64)
    for b in range(s["k"][0].shape[0]):
        s["k"][0][b] *= 30 if b % 3 == 0 else 0.1 if b % 3 == 1 else 1
    s["values"][0] = np.nan_to_num(f64(s["k"][0]))
    check(s, call(s, True), True)
    s["q"] = s["q"] * -1
    check(s, call(s, False), False)


def test_many_sequences():
    r = np.random.default_rng(0)
    lens = r.integers(0, 60, 400)
    new = np.minimum(r.integers(0, 5, 400), lens)
    s = chunk(lens.tolist(), new.tolist(), 8, 2, 64)
    check(s, call(s, True), True)


def test_rows_that_see_nothing():
    """More new rows than stored tokens: the first ones have a limit of 0 or less."""
    s = chunk([10, 0, 200], [30, 5, 200], 8, 2, 64)
    check(s, call(s, True), True)


def test_mass_forms_and_repeats():
    s = chunk([400, 90], [100, 90], 8, 2, 128)
    mass = call(s, True, mass_in=None, carry=3.0)
    check(s, mass, True, mass_in=None)
    own = s["mass_in"].clone()
    call(s, True, mass_in=own, carry=1.0, mass=own)
    for a, n in enumerate(s["lens"]):
        torch.testing.assert_close(own[a, :n], s["mass_in"][a, :n] + mass[a, :n], rtol=2.0 ** -22, atol=1e-38)
        assert torch.equal(own[a, n:], s["mass_in"][a, n:])
    for _ in range(3):
        assert torch.equal(call(s, True, mass_in=None), mass)


def test_one_row_each_agrees_with_decoding():
    s = chunk([900, 33, 2000], [1, 1, 1], 16, 2, 128)
    mass = call(s, True, mass_in=None)
    out, m2 = torch.empty(3, 16, 128, device=DEV), torch.full_like(mass, -3.0)
    ws = workspace(K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MASS, 3, s["mb"], 16))
    K.kvs_decode_attn_mass(s["pool"], 0, s["q"].contiguous(), 16, i32(s["table"]), s["mb"], i32(s["lens"]), 3, s["scale"], out,
                           None, 1.0, m2, ws)
    torch.testing.assert_close(mass, m2, rtol=2e-5, atol=0)


def test_captured_and_replayed():
    s = chunk([600, 1200], [200, 40], 8, 2, 128)
    ws = workspace(K.kvs_extend_mass_workspace_size(s["pool"], s["T"], 2, s["mb"], 8))
    off, table, lens, mass = i32(s["off"]), i32(s["table"]), i32(s["lens"]), torch.full_like(s["mass_in"], -3.0)
    q = s["q"].contiguous()
    run = lambda: K.kvs_extend_mass(s["pool"], 0, q, s["T"], off, 8, table, s["mb"], lens, 2, True, s["scale"], s["mass_in"], 0.75, mass, ws)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        q.neg_()
        for _ in range(3):
            graph.replay()
        side.synchronize()
    s["q"] = q
    check(s, mass, True)


@pytest.mark.parametrize("hkv, hq", [(32, 32), (8, 40), (2, 16), (1, 12), (8, 8)])
def test_a_larger_step_needs_no_less_workspace(hkv, hq):
    slab = [torch.zeros(2, hkv, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    p = K.kvs_pool_create(1, hkv, 64, 16, K.KVS_DTYPE_BF16, 2, 4096, [slab[0]], [slab[1]])
    tokens, seqs, blocks = [0, 1, 2, 15, 33, 100, 255, 257, 1000, 4096, 8192, 30000, 200000], [1, 2, 3, 32, 33, 600, 4096], [1, 8, 9, 96, 500, 4096]
    size = np.array([[[K.kvs_extend_mass_workspace_size(p, t, n, b, hq) for b in blocks] for n in seqs] for t in tokens])
    for axis in range(3):
        assert (np.diff(size, axis=axis) >= 0).all(), "tokens sequences blocks".split()[axis]


def test_one_workspace_for_every_step():
    big = chunk([2500, 300, 40], [1500, 300, 40], 8, 2, 64, seed=1)
    ws = workspace(K.kvs_extend_mass_workspace_size(big["pool"], big["T"], 3, big["mb"], 8)).fill_(0xC3)
    for s in (big, chunk([2400, 290, 30], [20, 7, 1], 8, 2, 64, seed=2), chunk([2300], [200], 8, 2, 64, seed=3), chunk([17], [1], 8, 2, 64, seed=4)):
        check(s, call(s, True, ws=ws), True)


def test_bad_blocks_lengths_and_offsets():
    s = chunk([300, 200], [300, 9], 8, 2, 64)
    s["table"][0, 1] = s["cap"]
    K_before = s["values"][0]
    mass = call(s, False)
    assert K.kvs_pool_check(s["pool"]) == K.KVS_DEVERR_BLOCK_ID
    # a bad block counts as zero keys: one more block of zeros in the oracle's pool
    s["values"][0] = np.concatenate([K_before, np.zeros((1,) + K_before.shape[1:])])
    check(s, mass, False)
    s = chunk([100, 60], [100, 60], 8, 2, 64)
    s["off"] = np.array([0, 100, 99])
    mass = call(s, True)
    assert K.kvs_pool_check(s["pool"]) == K.KVS_DEVERR_JOB and (mass == -3).all()
    s = chunk([50, 3], [4, 3], 8, 2, 64)
    s["values"] = [np.nan_to_num(x) for x in s["values"]]
    s["lens"] = [50, -1]
    mass = call(s, False)
    check(s, mass, False, lens=[50, 0], flags=K.KVS_DEVERR_SEQ_LEN)


def test_refusals():
    s = chunk([40], [5], 8, 2, 64)
    mx = make("mx4", [40], 8, 2, 128)
    ws = workspace(K.kvs_extend_mass_workspace_size(s["pool"], 5, 1, s["mb"], 8))
    good = dict(pool=s["pool"], layer=0, q=s["q"], n_tokens=5, tok_off=i32(s["off"]), n_q_heads=8, block_table=i32(s["table"]),
                max_blocks=s["mb"], seq_len=i32(s["lens"]), n_seq=1, causal=True, scale=0.1, mass_in=s["mass_in"], carry=1.0,
                mass=torch.zeros_like(s["mass_in"]), ws=ws)
    K.kvs_extend_mass(**good)
    for change in (dict(pool=mx["pool"]), dict(layer=1), dict(n_q_heads=7), dict(scale=0.0), dict(scale=float("inf")), dict(causal=2),
                   dict(carry=float("nan")), dict(ws=ws[:64]), dict(ws=None), dict(mass=None), dict(q=s["q"].float()), dict(n_tokens=6),
                   dict(max_blocks=s["mb"] + 1), dict(mass_in=s["mass_in"][:, 1:]), dict(tok_off=i32(s["off"]).cpu())):
        with pytest.raises((K.KvsError, ValueError)):
            K.kvs_extend_mass(**{**good, **change})
    K.kvs_extend_mass(**{**good, "n_seq": 0})
    assert K.kvs_pool_check(s["pool"]) == 0
