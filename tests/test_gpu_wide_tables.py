"""Tables far wider than their sequences, as a serving loop allocates them for the longest context: the forms that go by the
width of a table, and the space behind the sequences."""
import pytest

import test_gpu_compact as C
import test_gpu_decode_mass as D
import test_gpu_extend_mass as X

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, hq, hkv, d", [("bf16", 8, 2, 64), ("bf16", 16, 1, 128), ("mx4", 8, 2, 128)])
@pytest.mark.parametrize("lens, wider", [([300, 1, 0, 700], 8192), ([90] * 70, 600)])
def test_decode(kind, hq, hkv, d, lens, wider):
    s = D.make(kind, lens, hq, hkv, d, seed=wider, mb_extra=wider)
    D.check(s, *D.call(s))


@pytest.mark.parametrize("lens, new, hq, hkv, d", [
    ([300], [64], 8, 2, 128), ([300, 40, 0, 7], [4, 1, 0, 2], 16, 2, 128), ([900, 500], [900, 20], 8, 8, 64), ([33] * 40, [2] * 40, 8, 2, 64)])
@pytest.mark.parametrize("wider", [70, 500, 8192])
def test_chunks(monkeypatch, lens, new, hq, hkv, d, wider):
    monkeypatch.setattr(X, "make", lambda *a, **k: D.make(*a, **k, mb_extra=wider))
    s = X.chunk(lens, new, hq, hkv, d, seed=len(lens), pad=1)
    for causal in (True, False):
        X.check(s, X.call(s, causal), causal)


@pytest.mark.parametrize("kind, lens, shared", [("bf16", [300, 384, 0, 321], [0, 18, 0, 5]), ("bf16", [6000, 4000], [0, 100]),
                                                ("mx4", [700, 64], [0, 1]), ("bf16", [50] * 12, [0, 3] * 6)])
@pytest.mark.parametrize("wider", [520, 1100, 2100, 4100, 8192])   # one to eight CTAs a sequence, one launch and two
def test_choice_and_compaction(monkeypatch, kind, lens, shared, wider):
    state = C.state
    monkeypatch.setattr(C, "state", lambda r, lens, block, shared, cap_extra: state(r, lens, block, shared, cap_extra, mb_extra=wider))
    C.run_compact(kind, 2, 2, 128, lens, 0.4, shared, True)
    block = 16 if kind == "bf16" else 64
    pool, _, _ = C.make_pool(kind, 1, 1, 128, 2, len(lens))
    mb = -(-max(lens) // block) + wider
    mass = C.np.random.default_rng(wider).random((len(lens), mb * block)).astype(C.np.float32)
    budget = [x // 3 for x in lens]
    want, off = C.OC.keep_heavy(mass, lens, budget, 2, 9)
    idx, got = C.keep(pool, mass, lens, budget, 2, 9, mb)
    assert got.tolist() == off.tolist() and idx[: len(want)].tolist() == want.tolist() and (idx[len(want):] == -7).all()
    assert C.K.kvs_pool_check(pool) == 0
