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
