"""kvs_keep_heavy and kvs_compact against the host rules: every result is exact."""
import numpy as np
import pytest
import torch

from oracle import compact as OC
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, i64, workspace

pytestmark = pytest.mark.gpu


def make_pool(kind, layers, hkv, d, cap, n_seq, seed=0):
    """(pool, slabs in the order of a block's record, block tokens): bytes of any value."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = {"bf16": 16, "q4": 256, "mx4": 64}[kind]
    rnd = lambda w: torch.randint(0, 256, (cap, hkv, block, w), generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    if kind == "bf16":
        ks, vs = [rnd(2 * d) for _ in range(layers)], [rnd(2 * d) for _ in range(layers)]
        pool = K.kvs_pool_create(layers, hkv, d, block, K.KVS_DTYPE_BF16, cap, n_seq, ks, vs)
        return pool, [x for pair in zip(ks, vs) for x in pair], block
    w, dt = (d // 16, K.KVS_DTYPE_Q4G64) if kind == "q4" else (d // 32, K.KVS_DTYPE_MX4)
    parts = [[rnd(d // 2), rnd(d // 2), rnd(w), rnd(w)] for _ in range(layers)]
    pool = K.kvs_pool_create(layers, hkv, d, block, dt, cap, n_seq, *[[p[i] for p in parts] for i in range(4)])
    return pool, [x for p in parts for x in p], block


def keep(pool, mass, lens, budget, first, recent, max_blocks):
    n = len(lens)
    idx = torch.full((max(1, int(np.sum(np.maximum(lens, 0)))) + 8,), -7, dtype=torch.int32, device=DEV)
    off = torch.full((n + 1,), -7, dtype=torch.int64, device=DEV)
    K.kvs_keep_heavy(pool, torch.as_tensor(mass, dtype=torch.float32, device=DEV), i32(lens), n, max_blocks, i32(budget), first,
                     recent, idx, off)
    return idx, off


@pytest.mark.parametrize("kind, lens, budget, first, recent", [
    ("bf16", [1, 0, 16, 17, 40], [1, 3, 4, 0, 40], 0, 0),
    ("bf16", [100, 333, 5, 64], [50, 100, 2, 63], 4, 16),
    ("bf16", [1024, 1025, 4096, 4095], [1, 1024, 4000, 100], 7, 0),
    ("bf16", [20000, 131, 16385, 9000], [1234, 0, 16384, 8999], 3, 77),
    ("q4", [1500, 256, 700], [600, 256, 699], 0, 31),
    ("bf16", [8000, 5000], [2000, 4999], 16, 256),
    ("bf16", [12000, 8193, 30], [3000, 8192, 1], 16, 256),
    ("bf16", [50000, 40000], [1000, 39999], 64, 1024),
    ("bf16", [150000], [70000], 11, 13),           # beyond what eight CTAs hold in registers
])
@pytest.mark.parametrize("values", ["spread", "ties", "signed"])
def test_keep_heavy(kind, lens, budget, first, recent, values):
    pool, _, block = make_pool(kind, 1, 1, 128, 2, len(lens))
    mb = -(-max(lens) // block) + 1
    r = np.random.default_rng(len(lens) + max(lens))
    shape = (len(lens), mb * block)
    mass = {"spread": lambda: np.exp(3 * r.standard_normal(shape)), "ties": lambda: r.integers(0, 4, shape) * 0.25,
            "signed": lambda: np.where(r.random(shape) < 0.1, r.choice([np.nan, np.inf, -np.inf, -0.0, 0.0], shape),
                                       r.standard_normal(shape))}[values]().astype(np.float32)
    for a, n in enumerate(lens):
        mass[a, n:] = np.nan if a % 2 else np.inf   # behind the end: not looked at
    want, woff = OC.keep_heavy(mass, lens, budget, first, recent)
    idx, off = keep(pool, mass, lens, budget, first, recent, mb)
    assert off.tolist() == woff.tolist()
    np.testing.assert_array_equal(idx.cpu().numpy()[: len(want)], want)
    assert (idx[len(want):] == -7).all()
    assert K.kvs_pool_check(pool) == 0


def test_keep_heavy_clamps_a_bad_length():
    pool, _, _ = make_pool("bf16", 1, 1, 64, 2, 3)
    idx, off = keep(pool, np.ones((3, 32), np.float32), [40, -2, 3], [40, 5, 2], 0, 0, 2)
    assert off.tolist() == [0, 32, 32, 34] and idx[32:34].tolist() == [0, 1]
    assert K.kvs_pool_check(pool) == K.KVS_DEVERR_SEQ_LEN


def state(r, lens, block, shared, cap_extra, mb_extra=1):
    """A table of shuffled blocks; sequence a shares its first shared[a] blocks with the one before it."""
    n = len(lens)
    nb = [-(-x // block) for x in lens]
    mb = max(max(nb), 1) + mb_extra
    cap = sum(nb) + cap_extra
    ids = r.permutation(cap)
    table, at = np.full((n, mb), -1), 0
    refs = np.zeros(cap, np.int32)
    for a in range(n):
        s = min(shared[a], nb[a], nb[a - 1]) if a else 0
        table[a, :s] = table[a - 1, :s]
        table[a, s:nb[a]] = ids[at:at + nb[a] - s]
        at += nb[a] - s
        refs[table[a, :nb[a]]] += 1
    free = [int(x) for x in np.sort(ids[at:])[::-1]]
    return table, refs, free, mb, cap


CASES = [
    # kind, layers, heads, head_dim, lengths, share, fraction kept, blocks shared with the sequence before
    ("bf16", 1, 1, 64, [1, 5, 16, 17], 0.6, [0, 0, 0, 0]),
    ("bf16", 2, 2, 64, [300, 384, 0, 321], 0.4, [0, 0, 0, 0]),
    ("bf16", 2, 2, 128, [300, 384, 290, 321], 0.4, [0, 18, 18, 10]),
    ("bf16", 1, 3, 128, [2000, 2100, 1900], 0.95, [0, 50, 119]),
    ("bf16", 3, 1, 128, [5000], 0.3, [0]),
    ("bf16", 1, 2, 64, [4000, 4000], 0.5, [0, 250]),
    ("q4", 2, 2, 128, [1000, 257, 2049], 0.5, [0, 1, 0]),
    ("q4", 1, 2, 128, [3000, 3000], 0.9, [0, 0]),
]


@pytest.mark.parametrize("kind, layers, hkv, d, lens, part, shared", CASES)
@pytest.mark.parametrize("with_mass", [True, False])
def test_compact_with_room(kind, layers, hkv, d, lens, part, shared, with_mass):
    """The same with a free stack that serves every shared block."""
    run_compact(kind, layers, hkv, d, lens, part, shared, with_mass, cap_extra=500)


@pytest.mark.parametrize("kind, layers, hkv, d, lens, part, shared", CASES)
@pytest.mark.parametrize("with_mass", [True, False])
def test_compact(kind, layers, hkv, d, lens, part, shared, with_mass):
    run_compact(kind, layers, hkv, d, lens, part, shared, with_mass)


def run_compact(kind, layers, hkv, d, lens, part, shared, with_mass, cap_extra=40, lists=None, refs_change=None, flags=0, stream=None):
    r = np.random.default_rng(sum(lens) + hkv)
    block = {"bf16": 16, "q4": 256, "mx4": 64}[kind]
    table, refs, free, mb, cap = state(r, lens, block, shared, cap_extra)
    pool, slabs, _ = make_pool(kind, layers, hkv, d, cap, len(lens))
    lists = lists or [np.sort(r.permutation(x)[: int(np.ceil(part * x))]) for x in lens]
    idx, off = np.concatenate(lists), np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    mass = r.random((len(lens), mb * block)).astype(np.float32) if with_mass else None
    if refs_change:
        refs_change(refs, table)
    want = OC.compact([s.cpu().numpy() for s in slabs], table, lens, idx, off, mass, refs, free, block)
    dev = dict(table=i32(table), seq_len=i32(lens), refcount=i32(refs),
               free_ids=i32(np.concatenate([free, np.full(cap - len(free), -9)])), n_free=i32([len(free)]))
    md = None if mass is None else torch.as_tensor(mass, device=DEV)
    di, do = i32(np.concatenate([idx, [0]])), i64(off)
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_COMPACT, len(lens), mb))
    ws.fill_(0xAB)     # whatever was there
    torch.cuda.synchronize()
    K.kvs_compact(pool, dev["table"], mb, dev["seq_len"], len(lens), di, do, dev["refcount"], dev["free_ids"], dev["n_free"], ws,
                  mass=md, stream=stream)
    torch.cuda.synchronize()
    # the rules say who is left alone: with good lists that is a free stack too short for a sequence's shared blocks
    assert K.kvs_pool_check(pool) == (flags or (K.KVS_DEVERR_CAPACITY if want[6] else 0))
    w_slabs, w_table, w_len, w_mass, w_refs, w_free, _ = want
    np.testing.assert_array_equal(dev["table"].cpu().numpy(), w_table)
    np.testing.assert_array_equal(dev["seq_len"].cpu().numpy(), w_len)
    np.testing.assert_array_equal(dev["refcount"].cpu().numpy(), w_refs)
    assert int(dev["n_free"]) == len(w_free) and dev["free_ids"][: len(w_free)].tolist() == w_free
    if mass is not None:
        np.testing.assert_array_equal(md.cpu().numpy(), w_mass)
    for got, exp in zip(slabs, w_slabs):
        np.testing.assert_array_equal(got.cpu().numpy(), exp)


def test_compact_nothing_moves_and_everything_goes():
    """A prefix, the whole, and an empty list: no row is written."""
    run_compact("bf16", 1, 2, 64, [100, 64, 90, 33], 0, [0, 3, 2, 0], True,
                lists=[np.arange(37), np.arange(64), np.arange(0), np.arange(32)])


def test_compact_one_token_from_far():
    run_compact("bf16", 1, 1, 64, [3000, 3000, 3000], 0, [0, 0, 0], True,
                lists=[np.array([2999]), np.arange(1, 3000), np.concatenate([np.arange(1500), np.arange(1501, 3000)])])


def test_compact_leaves_bad_lists_alone():
    run_compact("bf16", 1, 1, 64, [64, 64, 64, 64], 0, [0, 0, 0, 0], True, flags=K.KVS_DEVERR_JOB,
                lists=[np.array([1, 5, 5]), np.array([3, 2]), np.array([0, 64]), np.array([1, 2, 63])])


def test_compact_short_free_stack():
    """Sequences take their blocks in turn (3, 5, 2 and 10 of the 5 that are free); one that finds too few stays as it
    is, a later one may still fit."""
    run_compact("bf16", 1, 1, 64, [160, 160, 160, 160], 0, [0, 10, 10, 10], True, cap_extra=-25, flags=K.KVS_DEVERR_CAPACITY,
                lists=[np.arange(1, 49), np.arange(1, 81), np.arange(3, 20), np.arange(5, 160)])


def test_compact_many_sequences():
    r = np.random.default_rng(5)
    lens = r.integers(0, 200, 1500).tolist()
    run_compact("bf16", 1, 1, 64, lens, 0.5, [3] * 1500, True, cap_extra=9000)


def test_compact_captured_and_replayed():
    """The call in a CUDA graph: replays begin from restored state, on another stream."""
    r = np.random.default_rng(1)
    lens, block, hkv, d = [500, 700], 16, 2, 64
    table, refs, free, mb, cap = state(r, lens, block, [0, 20], 60)
    pool, slabs, _ = make_pool("bf16", 1, hkv, d, cap, 2)
    first = [s.clone() for s in slabs]
    mass = r.random((2, mb * block)).astype(np.float32)
    idx, off = OC.keep_heavy(mass, lens, [200, 300], 4, 16)
    want = OC.compact([s.cpu().numpy() for s in slabs], table, lens, idx, off, mass, refs, free, block)
    start = dict(table=i32(table), seq_len=i32(lens), refcount=i32(refs),
                 free_ids=i32(np.concatenate([free, np.zeros(cap - len(free))])), n_free=i32([len(free)]),
                 mass=torch.as_tensor(mass, device=DEV))
    now = {k: v.clone() for k, v in start.items()}
    di, do = torch.zeros(600, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    budget, ws = i32([200, 300]), workspace(K.kvs_workspace_size(pool, K.KVS_OP_COMPACT, 2, mb))

    def step():
        for k in now:
            now[k].copy_(start[k])
        for s, x in zip(slabs, first):
            s.copy_(x)
        K.kvs_keep_heavy(pool, now["mass"], now["seq_len"], 2, mb, budget, 4, 16, di, do)
        K.kvs_compact(pool, now["table"], mb, now["seq_len"], 2, di, do, now["refcount"], now["free_ids"], now["n_free"], ws,
                      mass=now["mass"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            step()
        for _ in range(3):
            g.replay()
        side.synchronize()
    assert K.kvs_pool_check(pool) == 0
    np.testing.assert_array_equal(now["table"].cpu().numpy(), want[1])
    np.testing.assert_array_equal(now["mass"].cpu().numpy(), want[3])
    assert now["free_ids"][: int(now["n_free"])].tolist() == want[5]
    for got, exp in zip(slabs, want[0]):
        np.testing.assert_array_equal(got.cpu().numpy(), exp)
