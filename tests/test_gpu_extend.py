"""GPU attention of query chunks (prompt chunks, drafts, cross attention)
against the fp64 oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from oracle import attention as OA, extend as OE
import harness as H

DEV = H.DEV


def randn(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Batch:
    """Sequences of given new rows and lengths; groups share their leading
    `prefix` tokens (whole blocks).  Blocks behind a sequence's last token and
    rows of the last block behind it hold NaN.  The pool takes the planned path
    for every call; check() runs the library's own choice too (small calls: one
    launch without a plan)."""

    def __init__(self, new, lens, hq, hkv, d, prefix=0, groups=None, seed=0, pad=0, qscale=1.0):
        self.new, self.lens = np.array(new), np.array(lens)
        self.n = len(new)
        self.off = np.concatenate([[0], np.cumsum(self.new)])
        self.T = int(self.off[-1]) + pad
        need = -(-self.lens // 16)
        self.mb = int(max(need.max(), 1)) + 2
        groups = [0] * self.n if groups is None else groups
        prefix = [prefix] * (max(groups) + 1) if np.isscalar(prefix) else prefix
        r = np.random.default_rng(seed)
        cap = int(need.sum() + sum(p // 16 for p in prefix)) + 2
        ids = list(r.permutation(cap))
        bad = ids.pop()
        self.table = np.full((self.n, self.mb), -1)
        heads = [[ids.pop() for _ in range(p // 16)] for p in prefix]
        for a in range(self.n):
            for b in range(need[a]):
                self.table[a, b] = heads[groups[a]][b] if b < len(heads[groups[a]]) else ids.pop()
        self.table[:, need.max() if self.n else 0:] = bad    # a block of NaN behind the end
        self.k, self.v = randn(seed + 1, cap, hkv, 16, d), randn(seed + 2, cap, hkv, 16, d)
        self.k[bad] = self.v[bad] = float("nan")
        for a in range(self.n):
            e = int(self.lens[a])
            if e % 16 and (self.table == self.table[a, e // 16]).sum() == 1:
                self.k[self.table[a, e // 16], :, e % 16:] = float("nan")
                self.v[self.table[a, e // 16], :, e % 16:] = float("inf")
        self.q = (qscale * randn(seed + 3, self.T, hq, d).float()).to(torch.bfloat16)
        self.hq, self.hkv, self.d = hq, hkv, d
        self.pool = K.kvs_pool_create(1, hkv, d, 16, K.KVS_DTYPE_BF16, cap, max(self.n, 1), [self.k], [self.v])
        self.scale = d ** -0.5
        K.kvs_pool_set_test_flags(self.pool, K.KVS_TEST_EXTEND_PLANNED)

    def dev(self):
        return H.i32(self.off), H.i32(self.table), H.i32(self.lens)

    def ws(self):
        return torch.full((K.kvs_extend_workspace_size(self.pool, self.T, self.n, self.mb, self.hq),), 255,
                          dtype=torch.uint8, device=DEV)

    def run(self, causal, q=None, ws=None):
        off, tab, lens = self.dev()
        out = torch.full((self.T, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        K.kvs_extend_attn(self.pool, 0, self.q if q is None else q, self.T, off, self.hq, tab, self.mb, lens, self.n,
                          causal, self.scale, out, self.ws() if ws is None else ws)
        torch.cuda.synchronize()
        assert K.kvs_pool_check(self.pool) == 0
        return out

    def check(self, causal, out=None):
        if out is None:
            K.kvs_pool_set_test_flags(self.pool, 0)
            self.check(causal, self.run(causal))
            K.kvs_pool_set_test_flags(self.pool, K.KVS_TEST_EXTEND_PLANNED)
            out = self.run(causal)
        k, v = np.nan_to_num(f64(self.k), posinf=0.0), np.nan_to_num(f64(self.v), posinf=0.0)
        exp, mag, big = OE.extend_attention(f64(self.q), k, v, self.table, self.off, self.lens, 16, self.scale, causal)
        rows = ~np.isnan(exp[:, 0, 0])
        assert_attention(f64(out)[rows], exp[rows], mag[rows], big, self.d)
        assert (out[torch.from_numpy(~rows).to(DEV)] == 7).all()      # rows of no sequence
        return out


def assert_attention(got, exp, mag, big, d):
    """Half a bf16 step for the output and one for each weight P (2^-8 of the
    result, 2^-8 of sum p |V|), and what float32 adds to the exponents: a dot
    product of d terms is off by at most (d + 4) 2^-24 of sum |q k|, which moves
    a weight (and their sum) by twice that; 2^-20 covers ex2, the sums and the
    join of parts."""
    eps = 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 * (1 + 2.0 ** -8) + eps) * mag + 1e-30
    assert np.isfinite(got).all()
    bad = np.abs(got - exp) > tol
    assert not bad.any(), f"{bad.sum()} off, most {np.abs(got - exp).max():.3e} at {np.argwhere(bad)[0]}"
    # and on the whole as a bf16 result is: roundings are independent
    if exp.size >= 4096 and np.linalg.norm(exp) > 0:
        rel = np.linalg.norm(got - exp) / np.linalg.norm(exp)
        assert rel < 2.0 ** -8, rel


HEADS = [(8, 2, 64), (16, 2, 128), (4, 4, 128), (10, 2, 128), (12, 1, 64), (16, 1, 128), (6, 2, 64)]


@pytest.mark.parametrize("hq, hkv, d", HEADS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new, lens", [
    ([1], [1]), ([1], [17]), ([5], [5]), ([3, 1, 7], [129, 128, 127]), ([0, 4, 0], [30, 260, 0]), ([20], [300]),
])
def test_small(hq, hkv, d, causal, new, lens):
    Batch(new, lens, hq, hkv, d, seed=hq).check(causal)


@pytest.mark.parametrize("hq, hkv, d", HEADS[:4])
@pytest.mark.parametrize("causal", [True, False])
def test_long_ragged(hq, hkv, d, causal):
    """Many tiles and pieces, ends inside blocks and tiles, a padded batch."""
    Batch([130, 1, 257, 64, 9], [1111, 2000, 257, 400, 9], hq, hkv, d, seed=3, pad=5).check(causal)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(causal):
    """Empty contexts, and chunks longer than their sequence (the first rows
    see nothing): zeros."""
    b = Batch([4, 6, 300, 2], [0, 3, 40, 900], 8, 2, 64, pad=1)
    out = b.check(causal)
    assert (out[:4] == 0).all()
    if causal:
        assert (out[4:7] == 0).all() and (out[10:270] == 0).all()


@pytest.mark.parametrize("hq, hkv, d", [(16, 2, 128), (10, 2, 128), (8, 2, 64), (4, 4, 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new, own, prefix, groups", [
    ([1] * 9, [5] * 9, 512, None),                                      # drafts of one family
    ([3, 1, 4, 1, 5, 9, 2, 6], [0, 10, 200, 17, 1, 90, 300, 33], 640, None),
    ([2] * 12, [20] * 12, [256, 1024], [0] * 5 + [1] * 7),              # two families
    ([2] * 6, [20, 40, 60, 80, 100, 120], [256, 128], [0, 1, 0, 1, 0, 1]),  # no neighbours in common
    ([1, 0, 1, 1], [9, 9, 9, 9], 256, None),                            # one without rows
    ([40, 50, 60], [300, 200, 100], 768, None),                         # several units
])
def test_shared_prefix(hq, hkv, d, causal, new, own, prefix, groups):
    gr = [0] * len(new) if groups is None else groups
    pf = [prefix] * (max(gr) + 1) if np.isscalar(prefix) else prefix
    lens = [pf[g] + o + n for g, o, n in zip(gr, own, new)]
    b = Batch(new, lens, hq, hkv, d, prefix=prefix, groups=gr, seed=5, qscale=2.0)
    out = b.check(causal)
    # the same rows with every block stored apart
    apart = Batch(new, lens, hq, hkv, d, seed=5)
    apart.q = b.q
    for a in range(b.n):
        n = -(-lens[a] // 16)
        src, dst = torch.from_numpy(b.table[a, :n]).to(DEV), torch.from_numpy(apart.table[a, :n]).to(DEV)
        apart.k[dst], apart.v[dst] = b.k[src], b.v[src]
    alone = apart.run(causal)
    rows = f64(alone)
    # two results within their roundings of the same value
    assert np.abs(f64(out) - rows).max() <= 2.0 ** -6 * np.abs(rows).max()


def test_whole_prefix_shared_cross_attention():
    """States shared to the last key: no part of a sequence's own remains."""
    Batch([1, 2, 3, 1], [256] * 4, 8, 2, 128, prefix=256).check(False)
    Batch([1, 2, 3, 1], [250] * 4, 8, 2, 128, prefix=256).check(False)


def test_scores_that_climb():
    """Keys whose level jumps between tiles, up and down: the reference point
    moves in some tiles and stays in others."""
    b = Batch([70, 3], [1500, 900], 8, 2, 64, qscale=3.0)
    for a in range(2):
        for i in range(-(-int(b.lens[a]) // 16)):
            b.k[b.table[a, i]] *= float([0.1, 3.0, 1.0, 6.0, 0.5][(i // 8) % 5])
    b.check(True)
    b.check(False)


def test_large_scores_do_not_overflow():
    b = Batch([5], [400], 4, 4, 128, qscale=64.0)
    b.k *= 16
    out = b.run(True)
    assert torch.isfinite(out.float()).all()


def test_same_call_same_bits():
    b = Batch([9, 40, 3, 77], [3000, 2500, 2100, 2077], 16, 2, 128, prefix=2048, seed=8)
    ws = b.ws()
    a = b.run(True, ws=ws)
    for _ in range(3):
        assert torch.equal(a, b.run(True, ws=ws))


def test_many_sequences():
    """More sequences than one round of the plan's scan, some without rows."""
    r = np.random.default_rng(0)
    new = r.integers(0, 3, 1500)
    lens = new + r.integers(0, 40, 1500)
    Batch(new, lens, 4, 1, 64, seed=2).check(True)


@pytest.mark.parametrize("hkv, n, prefix", [(1, 700, 384), (2, 600, 256), (4, 300, 640)])
def test_many_sequences_over_one_prefix(hkv, n, prefix):
    """Families larger than the plan keeps in shared memory, and calls with so
    many units that nothing is split."""
    r = np.random.default_rng(n)
    new = r.integers(0, 3, n)
    new[:5] = 2
    lens = prefix + r.integers(0, 30, n) + new
    b = Batch(new, lens, 4 * hkv, hkv, 64, prefix=prefix, seed=2)
    out = b.run(True)
    rows = r.choice(np.nonzero(np.diff(b.off) > 0)[0], 60, replace=False)
    check_sequences(b, out, rows, True)


def check_sequences(b, out, seqs, causal):
    k, v = f64(b.k), f64(b.v)
    for a in seqs:
        t0, t1, n = b.off[a], b.off[a + 1], int(b.lens[a])
        ids = b.table[a, : -(-n // 16)]
        kk, vv = np.nan_to_num(k[ids], posinf=0.0), np.nan_to_num(v[ids], posinf=0.0)
        exp, mag, big = OE.extend_attention(f64(b.q[t0:t1]), kk, vv, np.arange(len(ids))[None], [0, t1 - t0], [n], 16,
                                            b.scale, causal)
        assert_attention(f64(out[t0:t1]), exp, mag, big, b.d)


@pytest.mark.parametrize("hq, hkv, d, new, n", [(1, 1, 128, 1, 40000), (8, 8, 64, 2, 24000), (12, 1, 64, 3, 33333)])
@pytest.mark.parametrize("causal", [True, False])
def test_one_long_context(hq, hkv, d, new, n, causal):
    """Few rows over a long context: more parts than a warp joins at a time."""
    b = Batch([new], [n], hq, hkv, d, seed=4)
    check_sequences(b, b.run(causal), [0], causal)


def test_a_call_too_large_for_parts():
    """So many rows that nothing is split or shared; sampled rows."""
    hq, hkv, d, n, prefix = 64, 4, 64, 4, 512
    new = [2100, 2200, 2050, 2077]
    b = Batch(new, [prefix + m + 100 for m in new], hq, hkv, d, prefix=prefix, seed=6)
    assert b.T * hq > 1 << 19
    out = b.run(True)
    k, v = np.nan_to_num(f64(b.k), posinf=0.0), np.nan_to_num(f64(b.v), posinf=0.0)
    q, o = f64(b.q), f64(out)
    r = np.random.default_rng(1)
    for t in r.integers(0, b.T, 24):
        a = int(np.searchsorted(b.off, t, side="right") - 1)
        lim = int(b.lens[a] - b.new[a] + (t - b.off[a]) + 1)
        ids = b.table[a, : -(-lim // 16)]
        for h in r.integers(0, hq, 3):
            exp, mag, big = OE.extend_attention(q[t:t + 1, h:h + 1], k[ids][:, h // 16:h // 16 + 1], v[ids][:, h // 16:h // 16 + 1],
                                                np.arange(len(ids))[None], [0, 1], [lim], 16, b.scale, True)
            assert_attention(o[t:t + 1, h:h + 1], exp, mag, big, d)


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    """Batches drawn over the whole range: groups, prefixes, empty sequences,
    lengths that end anywhere, padded rows."""
    r = np.random.default_rng(1000 + seed)
    hkv = int(r.choice([1, 2, 3]))
    hq = hkv * int(r.choice([1, 2, 3, 4, 5, 7, 8, 16]))
    d = int(r.choice([64, 128]))
    n = int(r.integers(1, 14))
    fams = int(r.integers(1, 4))
    groups = np.sort(r.integers(0, fams, n)).tolist()
    prefix = [16 * int(x) for x in r.integers(0, 40, fams)]
    new = r.integers(0, int(r.choice([2, 9, 90])), n)
    own = r.integers(0, int(r.choice([3, 200, 900])), n)
    lens = [max(0, prefix[g] * int(r.random() < 0.9) + int(o) + int(m) - int(r.integers(0, 3))) for g, o, m in zip(groups, own, new)]
    b = Batch(new, lens, hq, hkv, d, prefix=prefix, groups=groups, seed=seed, pad=int(r.integers(0, 4)),
              qscale=float(r.choice([0.5, 2.0, 6.0])))
    if b.T:
        b.check(bool(r.random() < 0.6))


def test_two_graphs_share_a_workspace():
    """Two captured calls of different batches and forms on one workspace,
    replayed in turn."""
    a = Batch([4, 9, 2, 30], [700, 650, 600, 900], 8, 2, 64, prefix=512)
    c = Batch([1] * 7, [90, 1, 300, 40, 5, 77, 1200], 8, 2, 64, seed=9)
    ws = max((a.ws(), c.ws()), key=lambda w: w.numel())
    want = [a.run(True), c.run(False)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    keep = []
    for b, causal in ((a, True), (c, False)):
        off, tab, lens = b.dev()
        out = torch.full_like(want[len(outs)], 7.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, b.hq, tab, b.mb, lens, b.n, causal, b.scale, out, ws)
        graphs.append(g)
        outs.append(out)
        keep.append((off, tab, lens))
    for i in (0, 1, 1, 0, 1):
        outs[i].fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    assert K.kvs_pool_check(a.pool) == 0 and K.kvs_pool_check(c.pool) == 0


def test_query_rows_of_one_projection():
    b = Batch([5, 30], [50, 400], 8, 2, 128)
    rows = randn(9, b.T, 12, 128)
    rows[:, :8] = b.q
    assert torch.equal(b.run(True), b.run(True, q=rows[:, :8]))


def test_plan_serves_layers_graphs_and_streams():
    hq, hkv, d = 16, 2, 128
    b = Batch([4, 9, 2, 30], [700, 650, 600, 900], hq, hkv, d, prefix=512)
    k2, v2 = randn(31, *b.k.shape), randn(32, *b.v.shape)
    pool = K.kvs_pool_create(2, hkv, d, 16, K.KVS_DTYPE_BF16, b.k.shape[0], b.n, [b.k, k2], [b.v, v2])
    K.kvs_pool_set_test_flags(pool, K.KVS_TEST_EXTEND_PLANNED)
    off, tab, lens = b.dev()
    ws = b.ws()
    ref = b.run(True)
    K.kvs_extend_plan(pool, b.T, off, hq, tab, b.mb, lens, b.n, True, ws)
    outs = [torch.empty(b.T, hq, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for _ in range(2):
        for layer in range(2):
            K.kvs_extend_attn_planned(pool, layer, b.q, b.T, off, hq, tab, b.mb, lens, b.n, True, b.scale, outs[layer], ws)
    torch.cuda.synchronize()
    assert K.kvs_pool_check(pool) == 0
    assert torch.equal(outs[0], ref)
    other = Batch([4, 9, 2, 30], [700, 650, 600, 900], hq, hkv, d, prefix=512)
    other.k.copy_(k2)
    other.v.copy_(v2)
    other.check(True, out=outs[1])
    # captured, then replayed with other queries and another step's lengths
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    q, out = b.q.clone(), torch.empty_like(b.q)
    with torch.cuda.graph(graph, stream=side):
        K.kvs_extend_attn(pool, 0, q, b.T, off, hq, tab, b.mb, lens, b.n, True, b.scale, out, ws)
        K.kvs_extend_attn(pool, 1, q, b.T, off, hq, tab, b.mb, lens, b.n, True, b.scale, outs[1], ws)
    q.copy_(randn(77, *q.shape))
    lens -= 3
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert K.kvs_pool_check(pool) == 0
    b.q, b.lens = q, b.lens - 3
    with torch.cuda.stream(side):
        again = torch.empty_like(out)
        K.kvs_extend_attn(pool, 0, q, b.T, off, hq, tab, b.mb, lens, b.n, True, b.scale, again, ws)
    side.synchronize()
    assert torch.equal(out, again)
    b.check(True, out=out)


def test_plan_of_another_call_is_refused():
    b = Batch([4, 9], [70, 65], 8, 2, 64)
    off, tab, lens = b.dev()
    ws = b.ws()
    out = torch.full_like(b.q, 7.0)
    for planned in (False, True):
        if planned:
            K.kvs_extend_plan(b.pool, b.T, off, 8, tab, b.mb, lens, b.n, False, ws)
        K.kvs_extend_attn_planned(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, ws)
        torch.cuda.synchronize()
        assert K.kvs_pool_check(b.pool) == K.KVS_DEVERR_PLAN
        assert (out == 7).all()
    K.kvs_extend_plan(b.pool, b.T, off, 8, tab, b.mb, lens, b.n, True, ws)
    K.kvs_extend_attn_planned(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, out, ws)
    b.check(True, out=out)


@pytest.mark.parametrize("flags", [0, K.KVS_TEST_EXTEND_PLANNED])
def test_bad_tables_lengths_and_offsets_are_flagged(flags):
    b = Batch([4, 9], [70, 65], 8, 2, 64)
    K.kvs_pool_set_test_flags(b.pool, flags)
    out = b.run(True)
    good = b.table.copy()
    # unmapped and out-of-range ids count as zero keys and values
    for bad in (-1, b.k.shape[0]):
        b.table[0, 1] = bad
        off, tab, lens = b.dev()
        got = torch.full_like(b.q, 7.0)
        K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, got, b.ws())
        torch.cuda.synchronize()
        assert K.kvs_pool_check(b.pool) == K.KVS_DEVERR_BLOCK_ID
        assert torch.equal(got[4:], out[4:]) and torch.isfinite(got.float()).all() and not torch.equal(got[:4], out[:4])
        kz, vz = np.nan_to_num(f64(b.k), posinf=0.0), np.nan_to_num(f64(b.v), posinf=0.0)
        kz[good[0, 1]] = vz[good[0, 1]] = 0
        exp, mag, big = OE.extend_attention(f64(b.q), kz, vz, good, b.off, b.lens, 16, b.scale, True)
        assert_attention(f64(got), exp, mag, big, 64)
    b.table = good
    # lengths outside the table
    b.lens[1] = b.mb * 16 + 1
    off, tab, lens = b.dev()
    got = torch.full_like(b.q, 7.0)
    K.kvs_extend_attn(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, True, b.scale, got, b.ws())
    torch.cuda.synchronize()
    assert K.kvs_pool_check(b.pool) & K.KVS_DEVERR_SEQ_LEN
    assert torch.equal(got[:4], out[:4])
    # offsets
    for off_bad in ([0, 4, 14], [0, 5, 3], [-1, 4, 13], [4, 2, 13]):
        got = torch.full_like(b.q, 7.0)
        K.kvs_extend_attn(b.pool, 0, b.q, b.T, H.i32(off_bad), 8, tab, b.mb, H.i32([70, 65]), b.n, True, b.scale, got, b.ws())
        torch.cuda.synchronize()
        assert K.kvs_pool_check(b.pool) & K.KVS_DEVERR_JOB
        assert (got == 7).all()


@pytest.mark.parametrize("n, new, mb", [(32, 1, 96), (31, 3, 90), (1, 64, 96), (32, 0, 3), (7, 40, 95)])
@pytest.mark.parametrize("causal", [True, False])
def test_calls_of_one_launch(n, new, mb, causal):
    """The largest calls that run without a plan, and a plan that such a call
    does not need: the steps apart give the same bits."""
    r = np.random.default_rng(n)
    rows = np.full(n, new)
    rows[0] = max(new, 1)
    rows[n // 2:n // 2 + 1] += 1
    lens = np.maximum(r.integers(0, 16 * mb + 1, n), 0)
    lens[-1] = 16 * mb
    b = Batch(rows, lens, 8, 2, 64, seed=n)
    b.mb, b.table = mb, np.ascontiguousarray(b.table[:, :mb])
    K.kvs_pool_set_test_flags(b.pool, 0)
    before = K.kvs_launch_count()
    out = b.run(causal)
    assert K.kvs_launch_count() == before + 1
    b.check(causal, out)
    off, tab, lens = b.dev()
    ws, again = b.ws(), torch.full_like(out, 7.0)
    K.kvs_extend_plan(b.pool, b.T, off, 8, tab, b.mb, lens, b.n, causal, ws)
    assert (ws == 255).all()
    K.kvs_extend_attn_planned(b.pool, 0, b.q, b.T, off, 8, tab, b.mb, lens, b.n, causal, b.scale, again, ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("new, ctx, hq, hkv, d", [([1800, 900, 1300], [100, 0, 1111], 16, 4, 64), ([700, 64, 0, 1500], [0, 0, 50, 3], 8, 8, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_chunks_of_one_launch(new, ctx, hq, hkv, d, causal):
    """Chunks that fill the device without splits: several rounds of items over
    the CTAs, the same result on every call."""
    lens = [n + c for n, c in zip(new, ctx)]
    b = Batch(new, lens, hq, hkv, d, seed=3, pad=2)
    planned = b.run(causal)
    K.kvs_pool_set_test_flags(b.pool, 0)
    before = K.kvs_launch_count()
    out = b.run(causal)
    assert K.kvs_launch_count() == before + 1
    for _ in range(2):
        assert torch.equal(out, b.run(causal))
    assert (out[-2:] == 7).all()
    # two results within their roundings (P and output, 2^-8 each) of one value
    assert (out.float() - planned.float()).abs().max() <= 2.0 ** -6 * float(b.v[torch.isfinite(b.v)].abs().max())
    check_sequences(b, out, [len(new) - 3], causal)


@pytest.mark.parametrize("new, ctx, hq, hkv", [([2600], [77], 32, 32), ([900, 2000], [1000, 0], 40, 8), ([3500], [0], 24, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_chunks_against_sampled_rows(new, ctx, hq, hkv, causal):
    """Long chunks of head_dim 128 in one launch: several rounds, row tiles
    that end anywhere, key ends inside blocks, NaN behind them."""
    lens = [n + c for n, c in zip(new, ctx)]
    b = Batch(new, lens, hq, hkv, 128, seed=6, pad=3)
    planned = b.run(causal)
    K.kvs_pool_set_test_flags(b.pool, 0)
    before = K.kvs_launch_count()
    out = b.run(causal)
    assert K.kvs_launch_count() == before + 1
    assert torch.equal(out, b.run(causal))
    assert (out[-3:] == 7).all()
    # two results within their roundings (P and output, 2^-8 each) of one value
    assert (out.float() - planned.float()).abs().max() <= 2.0 ** -6 * float(b.v[torch.isfinite(b.v)].abs().max())
    k, v = np.nan_to_num(f64(b.k)), np.nan_to_num(f64(b.v), posinf=0.0)
    for a in range(len(new)):
        ids = b.table[a, : -(-int(b.lens[a]) // 16)]
        for j in [0, new[a] - 1, *np.random.default_rng(a).integers(0, new[a], 12)]:
            t, n = int(b.off[a]) + int(j), int(b.lens[a]) - new[a] + int(j) + 1 if causal else int(b.lens[a])
            exp, mag, big = OE.extend_attention(f64(b.q[t:t + 1]), k[ids], v[ids], np.arange(len(ids))[None], [0, 1], [n], 16,
                                                b.scale, False)
            assert_attention(f64(out[t:t + 1]), exp, mag, big, b.d)


def test_refusals():
    b = Batch([4, 9], [70, 65], 8, 2, 64)
    off, tab, lens = b.dev()
    out, ws = torch.empty_like(b.q), b.ws()

    def call(layer=0, q=b.q, hq=8, causal=True, scale=b.scale, ws=ws, n=b.n, mb=b.mb, out=out):
        K.kvs_extend_attn(b.pool, layer, q, b.T, off, hq, tab, mb, lens, n, causal, scale, out, ws)

    for kw in (dict(layer=1), dict(layer=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(ws=ws[:-1]), dict(ws=ws[1:]), dict(causal=2), dict(mb=0), dict(n=3),
               dict(q=b.q.float()), dict(q=b.q.half()), dict(hq=7), dict(out=out.transpose(0, 1))):
        with pytest.raises((K.KvsError, ValueError)):
            call(**kw)
    q40 = torch.zeros(b.T, 40, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(K.KvsError):
        K.kvs_extend_workspace_size(b.pool, b.T, b.n, b.mb, 40)          # 20 query heads per KV head
    with pytest.raises(K.KvsError):
        K.kvs_extend_attn(b.pool, 0, q40, b.T, off, 40, tab, b.mb, lens, b.n, True, 1.0, q40.clone(), ws)
    z8 = [torch.zeros(2, 2, 256, 64, dtype=torch.uint8, device=DEV) for _ in range(2)]
    z16 = [torch.zeros(2, 2, 256, 2, 2, dtype=torch.float16, device=DEV) for _ in range(2)]
    p4 = K.kvs_pool_create(1, 2, 128, 256, K.KVS_DTYPE_Q4G64, 2, 1, [z8[0]], [z8[1]], [z16[0]], [z16[1]])
    with pytest.raises(K.KvsError):
        K.kvs_extend_workspace_size(p4, 1, 1, 1, 8)
    assert K.kvs_pool_check(b.pool) == 0
    K.kvs_extend_attn(b.pool, 0, b.q, 0, off, 8, tab, b.mb, lens, b.n, True, 1.0, out, ws)   # nothing to do


def test_prompt_then_steps():
    """A prompt chunk and three decode steps as a model runs them: rotated
    append, chunk attention, single-token appends and decode attention, with
    the chunk attention of one row beside it."""
    hq, hkv, d, theta = 8, 2, 128, 1e6
    new, n = [37, 5, 130], 3
    lens = np.array(new)
    mb, cap = 12, 36
    table = np.random.default_rng(1).permutation(cap).reshape(n, mb)
    ks, vs = randn(1, cap, hkv, 16, d), randn(2, cap, hkv, 16, d)
    pool = K.kvs_pool_create(1, hkv, d, 16, K.KVS_DTYPE_BF16, cap, n, [ks], [vs])
    ax, tab = K.RopeAxes(theta, (64,)), H.i32(table)
    kh = [np.zeros((0, hkv, d))] * n
    vh = [np.zeros((0, hkv, d))] * n
    for step in range(4):
        m = np.array(new) if step == 0 else np.ones(n, int)
        if step:
            lens = lens + 1
        T, off = int(m.sum()), np.concatenate([[0], np.cumsum(m)])
        qkv = randn(10 + step, T, hq + 2 * hkv, d)
        q = torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV)
        K.kvs_append(pool, 0, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], T, H.i32(off), tab, mb, H.i32(lens), n, rope=ax,
                     q=qkv[:, :hq], n_q_heads=hq, q_out=q)
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(K.kvs_extend_workspace_size(pool, T, n, mb, hq), dtype=torch.uint8, device=DEV)
        K.kvs_extend_attn(pool, 0, q, T, H.i32(off), hq, tab, mb, H.i32(lens), n, True, d ** -0.5, out, ws)
        assert K.kvs_pool_check(pool) == 0
        kc, vc = torch.empty(T, hkv, d, dtype=torch.bfloat16, device=DEV), torch.empty(T, hkv, d, dtype=torch.bfloat16, device=DEV)
        K.kvs_gather(pool, 0, T, H.i32(off), tab, mb, H.i32(lens), n, kc, vc)
        for a in range(n):
            s = slice(off[a], off[a + 1])
            pos = np.arange(lens[a] - m[a], lens[a])[None]
            # exact rotation of the inputs; the stored key is its bf16 rounding
            ek = OE.rotate_axes(f64(qkv[s, hq:hq + hkv]), pos, theta, (64,))
            assert np.abs(f64(kc[s]) - ek).max() <= 2.0 ** -8 * np.abs(ek).max() + 1e-5
            kh[a], vh[a] = np.concatenate([kh[a], f64(kc[s])]), np.concatenate([vh[a], f64(qkv[s, hq + hkv:])])
            exp, mag, big = OE.extend_attention(f64(q[s]), kh[a][None].transpose(0, 2, 1, 3), vh[a][None].transpose(0, 2, 1, 3),
                                                np.zeros((1, 1), int), [0, m[a]], [lens[a]], int(lens[a]), d ** -0.5, True)
            assert_attention(f64(out[s]), exp, mag, big, d)
        if step:
            dec = torch.empty(n, hq, d, dtype=torch.float32, device=DEV)
            w2 = H.workspace(K.kvs_workspace_size(pool, K.KVS_OP_DECODE_ATTN, n, mb, hq))
            K.kvs_decode_attn(pool, 0, q, hq, tab, mb, H.i32(lens), n, None, None, None, theta, d ** -0.5, dec, w2)
            torch.cuda.synchronize()
            exp = OA.decode_attention(f64(q), f64(ks), f64(vs), table, lens, 16, d ** -0.5)
            H.assert_close_attn(f64(dec), exp)
            assert (np.abs(f64(out) - f64(dec)) <= 2.0 ** -7 * np.abs(f64(vs)).max()).all()
