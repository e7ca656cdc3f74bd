"""What kvs_compact does with inputs that belong to no pool: every case ends with a status bit and leaves a sequence that
cannot be moved as it was."""
import numpy as np
import pytest
import torch

from oracle import compact as OC
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, i64, workspace
from test_gpu_compact import make_pool, run_compact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("idle", [0, 30])     # one launch for check and tables, or two
def test_blocks_of_two_sequences_that_are_counted_once(idle):
    """The second sequence lists the first one's blocks, whose counts say 1: the rows of both are more than the pool
    holds, so the second is left as it was; the third, with blocks of its own, is compacted."""
    block, hkv, d, own, cap = 16, 1, 64, 240, 256
    pool, slabs, _ = make_pool("bf16", 1, hkv, d, cap, 3 + idle)
    table = np.full((3 + idle, own), -1)
    ids = np.random.default_rng(idle).permutation(cap)
    table[0], table[1], table[2, :2] = ids[:own], ids[:own], ids[own:own + 2]
    lens = [own * block, own * block, 2 * block] + [0] * idle
    refs = np.zeros(cap, np.int64)
    refs[table[table >= 0]] = 1
    lists = [np.arange(1, lens[0]), np.arange(1, lens[1]), np.arange(5, 20)] + [np.arange(0)] * idle
    assert len(lists[0]) + len(lists[1]) > cap * block
    mass = np.random.default_rng(1).random((3 + idle, own * block)).astype(np.float32)
    alone = [lists[0], np.array([1, 1]), *lists[2:]]     # the rule for a sequence that is left alone
    off = lambda ls: np.concatenate([[0], np.cumsum([len(x) for x in ls])])  # noqa: E731
    free = [int(x) for x in np.sort(ids[own + 2:])[::-1]]
    want = OC.compact([s.cpu().numpy() for s in slabs], table, lens, np.concatenate(alone), off(alone), mass, refs, free, block)
    got = dict(table=i32(table), lens=i32(lens), refs=i32(refs), free=i32(np.concatenate([free, np.zeros(cap - len(free))])),
               n_free=i32([len(free)]), mass=torch.as_tensor(mass, device=DEV))
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_COMPACT, 3 + idle, own)).fill_(0xAB)
    K.kvs_compact(pool, got["table"], own, got["lens"], 3 + idle, i32(np.concatenate(lists)), i64(off(lists)), got["refs"],
                  got["free"], got["n_free"], ws, mass=got["mass"])
    assert K.kvs_pool_check(pool) == K.KVS_DEVERR_REFCOUNT
    for name, exp in zip(("table", "lens", "mass", "refs"), want[1:5]):
        np.testing.assert_array_equal(got[name].cpu().numpy(), exp)
    assert got["free"][: int(got["n_free"])].tolist() == want[5]
    for x, exp in zip(slabs, want[0]):
        np.testing.assert_array_equal(x.cpu().numpy(), exp)


@pytest.mark.parametrize("kind, d, lens", [("bf16", 64, [700, 900]), ("bf16", 128, [5000, 300, 1200]), ("q4", 128, [2000, 600])])
def test_blocks_with_references_elsewhere(kind, d, lens):
    """Some blocks of every sequence are also referenced from outside: new blocks beside rows that move in place."""
    def more(refs, table):
        used = table[table >= 0]
        refs[used[np.random.default_rng(len(used)).random(len(used)) < 0.3]] += 1
    run_compact(kind, 2, 2, d, lens, 0.5, [0] * len(lens), True, cap_extra=200, refs_change=more)


@pytest.mark.parametrize("kind, hkv", [("bf16", 2), ("mx4", 1)])
def test_a_wait_that_runs_out_writes_nothing(kind, hkv):
    """The first item never says that it has read its first chain: the one item that writes where those rows lay leaves
    them, everything else moves, and the next call is whole."""
    d, rows = (64, 128) if kind == "bf16" else (128, 256)     # places of an item
    pool, slabs, block = make_pool(kind, 2, hkv, d, 8 * rows // 16, 1)
    cap, n, mb = 8 * rows // 16, 8 * rows, 8 * rows // block
    ids = np.random.default_rng(3).permutation(cap)
    table, refs, free = ids[None, :mb], np.zeros(cap, np.int64), [int(x) for x in ids[mb:]]
    refs[table] = 1
    lists = np.arange(rows, n)                                # item i reads where item i + 1 writes
    want = OC.compact([s.cpu().numpy() for s in slabs], table, [n], lists, [0, len(lists)], None, refs, free, block)
    was = [s.cpu().numpy() for s in slabs]
    args = (i32(lists), i64([0, len(lists)]))
    state = lambda: (i32(refs), i32(np.concatenate([free, np.zeros(cap - len(free))])), i32([len(free)]))  # noqa: E731
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_COMPACT, 1, mb)).fill_(0xAB)
    start = [s.clone() for s in slabs]
    K.kvs_pool_set_test_flags(pool, K.KVS_TEST_STALL_COMPACT)
    K.kvs_compact(pool, i32(table), mb, i32([n]), 1, *args, *state(), ws)
    assert K.kvs_pool_check(pool) == K.KVS_DEVERR_WAIT_TIMEOUT
    places = np.arange(rows, 2 * rows)
    for i, (x, exp) in enumerate(zip(slabs, want[0])):
        if i in ((0,) if kind == "bf16" else (0, 2)):         # the first chain: layer 0, keys (and their scales), head 0
            exp = exp.copy()
            exp[table[0, places // block], 0, places % block] = was[i][table[0, places // block], 0, places % block]
        np.testing.assert_array_equal(x.cpu().numpy(), exp)
    for x, y in zip(slabs, start):
        x.copy_(y)
    K.kvs_compact(pool, i32(table), mb, i32([n]), 1, *args, *state(), ws)
    assert K.kvs_pool_check(pool) == 0
    for x, exp in zip(slabs, want[0]):
        np.testing.assert_array_equal(x.cpu().numpy(), exp)


@pytest.mark.parametrize("lens, budget, cap, whole", [
    ([100, 333, 5, 64], [50, 100, 2, 63], 150, 2),      # the third does not fit
    ([100, 333, 5, 64], [50, 100, 2, 63], 151, 2),
    ([300], [-7], 20, 1),                                # protected tokens alone, as many as fit
    ([300], [-7], 19, 0),                                # they are more than a list of the budgets' sum
    ([64, 40], [64, 40], 64, 1),                         # everything is kept
    ([20000, 40], [1000, 40], 999, 0),                   # several CTAs a sequence
    ([20, 0], [0, 5], 0, 2),                             # an empty list, and no list
])
def test_a_list_that_is_too_short(lens, budget, cap, whole):
    """No index is written past the list; the compaction that gets it leaves those sequences as they were."""
    first, recent, n = (4, 16, len(lens)) if cap else (0, 0, len(lens))
    block, hkv, d = 16, 1, 64
    nb = [-(-x // block) for x in lens]
    mb, used = max(nb) + 1, sum(nb)
    pool, slabs, _ = make_pool("bf16", 1, hkv, d, used + 1, n)
    table, at = np.full((n, mb), -1), 0
    for a in range(n):
        table[a, :nb[a]] = np.arange(at, at + nb[a])
        at += nb[a]
    refs = (np.arange(used + 1) < used).astype(np.int64)
    mass = np.random.default_rng(sum(lens)).random((n, mb * block)).astype(np.float32)
    lists, off = OC.keep_heavy(mass, lens, budget, first, recent)
    memory = torch.full((len(lists) + 64,), -7, dtype=torch.int32, device=DEV)
    idx, do, md = memory[:cap], torch.full((n + 1,), -7, dtype=torch.int64, device=DEV), torch.as_tensor(mass, device=DEV)
    K.kvs_keep_heavy(pool, md, i32(lens), n, mb, i32(budget), first, recent, idx, do)
    fits = off[1:] <= cap
    assert K.kvs_pool_check(pool) == (0 if fits.all() else K.KVS_DEVERR_CAPACITY)
    assert do.tolist() == off.tolist() and fits[:whole].all() and not fits[whole:whole + 1].any()
    want = np.full(len(memory), -7)
    for a in np.nonzero(fits)[0]:
        want[off[a]:off[a + 1]] = lists[off[a]:off[a + 1]]
    np.testing.assert_array_equal(memory.cpu().numpy(), want)
    # and on: sequences whose offsets lead out of the list keep everything
    rule = [lists[off[a]:off[a + 1]] if fits[a] else np.array([1, 1]) for a in range(n)]
    roff = np.concatenate([[0], np.cumsum([len(x) for x in rule])])
    exp = OC.compact([s.cpu().numpy() for s in slabs], table, lens, np.concatenate(rule), roff, mass, refs, [used], block)
    t, ln, rc, free, nf = i32(table), i32(lens), i32(refs), i32([used] + [0] * used), i32([1])
    ws = workspace(K.kvs_workspace_size(pool, K.KVS_OP_COMPACT, n, mb)).fill_(0xAB)
    K.kvs_compact(pool, t, mb, ln, n, idx, do, rc, free, nf, ws, mass=md)
    assert K.kvs_pool_check(pool) == (0 if fits.all() else K.KVS_DEVERR_JOB)
    for got, x in zip((t, ln, md, rc), exp[1:5]):
        np.testing.assert_array_equal(got.cpu().numpy(), x)
    for x, y in zip(slabs, exp[0]):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
