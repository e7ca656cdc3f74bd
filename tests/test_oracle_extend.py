"""The oracle of the operators on new tokens, pinned without a GPU, and the
argument checks of the calls that need no pool."""
import ctypes

import numpy as np
import pytest

from oracle import attention as OA, extend as OE, rope as OR


def test_one_axis_is_the_plain_rotation():
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 3, 64))
    pos = np.array([[0, 1, 7, 100, 4000]])
    y = OE.rotate_axes(x, pos, 1e4, (32,))
    for t in range(5):
        np.testing.assert_allclose(y[t], OR.rotate(x[t], int(pos[0, t]), 1e4), atol=1e-11)


def test_axes_turn_their_own_pairs_and_come_back():
    r = np.random.default_rng(1)
    x = r.standard_normal((4, 2, 128))
    sec = (16, 24, 24)
    pos = r.integers(-5, 1 << 20, (3, 4))
    y = OE.rotate_axes(x, pos, 1e6, sec)
    np.testing.assert_allclose(OE.rotate_axes(y, pos, 1e6, sec, inverse=True), x, atol=1e-9)
    # moving one axis changes that axis' pairs alone
    pos2 = pos.copy()
    pos2[1] += 3
    z = OE.rotate_axes(x, pos2, 1e6, sec)
    same = np.abs(y - z).max(axis=(0, 1)) == 0
    want = np.ones(128, bool)
    want[16:40] = want[80:104] = False
    np.testing.assert_array_equal(same, want)


def test_own_spectrum_starts_again_on_every_axis():
    w, axis = OE.axes_frequencies(64, 1e4, (16, 16), own_spectrum=True)
    np.testing.assert_allclose(w[:16], w[16:])
    assert w[0] == 1.0 and axis.tolist() == [0] * 16 + [1] * 16
    w1, _ = OE.axes_frequencies(64, 1e4, (16, 16))
    assert np.all(np.diff(w1) < 0)


def test_last_row_of_a_chunk_is_a_decode_step():
    r = np.random.default_rng(2)
    kp, vp = r.standard_normal((6, 2, 16, 64)), r.standard_normal((6, 2, 16, 64))
    table = np.array([[4, 1, 3], [0, 2, -1]])
    off, lens = np.array([0, 5, 5]), np.array([37, 20])
    q = r.standard_normal((5, 4, 64))
    out, _, _ = OE.extend_attention(q, kp, vp, table, off, lens, 16, 0.125, True)
    ref = OA.decode_attention(q[4:5], kp, vp, table[:1], lens[:1], 16, 0.125)
    np.testing.assert_allclose(out[4], ref[0], atol=1e-12)
    ref = OA.decode_attention(q[0:1], kp, vp, table[:1], np.array([33]), 16, 0.125)
    np.testing.assert_allclose(out[0], ref[0], atol=1e-12)
    full, _, _ = OE.extend_attention(q, kp, vp, table, off, lens, 16, 0.125, False)
    ref = OA.decode_attention(q[0:1], kp, vp, table[:1], lens[:1], 16, 0.125)
    np.testing.assert_allclose(full[0], ref[0], atol=1e-12)


def test_rows_that_see_nothing_are_zero():
    r = np.random.default_rng(3)
    kp = r.standard_normal((2, 1, 16, 64))
    q = r.standard_normal((4, 1, 64))
    out, _, _ = OE.extend_attention(q, kp, kp, np.array([[1]]), [0, 4], [2], 16, 1.0, True)
    assert (out[:2] == 0).all() and (out[2:] != 0).any()


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from shared_paged_kv_gb300 import kvs as K
    return K.load()


def test_calls_refuse_a_null_pool(lib):
    from shared_paged_kv_gb300 import kvs as K
    sz = ctypes.c_size_t()
    bad = K.KVS_ERR_INVALID_ARG
    assert lib.kvs_append(None, 0, None, 128, None, 128, None, 0, 0, None, None, 1, None, None, None, 1, None, 1, None) == bad
    assert lib.kvs_gather(None, 0, None, 1, None, 1, None, 1, None, None, None) == bad
    assert lib.kvs_extend_workspace_size(None, 1, 1, 1, 1, ctypes.byref(sz)) == bad
    assert lib.kvs_extend_plan(None, None, 1, 1, None, 1, None, 1, 1, None, 0, None) == bad
    assert lib.kvs_extend_attn_planned(None, 0, None, 64, None, 1, 1, None, 1, None, 1, 1, 1.0, None, None, 0, None) == bad
    assert lib.kvs_extend_attn(None, 0, None, 64, None, 1, 1, None, 1, None, 1, 1, 1.0, None, None, 0, None) == bad


@pytest.mark.parametrize("change, status", [
    (dict(head_dim=96), "KVS_ERR_UNSUPPORTED"),
    (dict(n_tokens=-1), "KVS_ERR_INVALID_ARG"),
    (dict(n_heads=0), "KVS_ERR_INVALID_ARG"),
    (dict(x_stride=120), "KVS_ERR_INVALID_ARG"),
    (dict(x_stride=132), "KVS_ERR_INVALID_ARG"),
    (dict(out_stride=64), "KVS_ERR_INVALID_ARG"),
    (dict(x=None), "KVS_ERR_INVALID_ARG"),
    (dict(pos=None), "KVS_ERR_INVALID_ARG"),
    (dict(x=24), "KVS_ERR_INVALID_ARG"),
    (dict(out=4096, out_stride=256), "KVS_ERR_INVALID_ARG"),
    (dict(axes=(0.0, (32,))), "KVS_ERR_INVALID_ARG"),
    (dict(axes=(float("nan"), (32,))), "KVS_ERR_INVALID_ARG"),
    (dict(axes=(float("inf"), (32,))), "KVS_ERR_INVALID_ARG"),
    (dict(axes=(1e4, (31,))), "KVS_ERR_INVALID_ARG"),
    (dict(axes=(1e4, (33, -1))), "KVS_ERR_INVALID_ARG"),
    (dict(axes=None), "KVS_ERR_INVALID_ARG"),
    (dict(n_tokens=0), "KVS_OK"),
])
def test_rope_apply_refusals(lib, change, status):
    """Everything is refused on the host: nothing here reaches a device."""
    from shared_paged_kv_gb300 import kvs as K
    a = dict(x=4096, x_stride=128, pos=8192, axes=(1e4, (32,)), out=12288, out_stride=128, n_tokens=3, n_heads=2, head_dim=64)
    a.update(change)
    axes = None if a["axes"] is None else ctypes.byref(K.RopeAxes(*a["axes"]))
    got = lib.kvs_rope_apply(a["x"], a["x_stride"], a["pos"], axes, 0, a["out"], a["out_stride"], a["n_tokens"],
                             a["n_heads"], a["head_dim"], None)
    assert got == getattr(K, status)


def test_binding_checks_rows_and_sections():
    import torch
    from shared_paged_kv_gb300 import kvs as K
    with pytest.raises(ValueError):
        K.RopeAxes(1e4, ())
    with pytest.raises(ValueError):
        K.RopeAxes(1e4, (8, 8, 8, 8))
    ok = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    for bad in (ok.float(), ok.to(torch.float16), ok.to(torch.int32)):
        with pytest.raises(ValueError, match="bf16 rows"):
            K._rows(bad, 4, 6, 64, "x")
    with pytest.raises(ValueError, match="CUDA tensor"):
        K._rows(ok, 4, 6, 64, "x")
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="contiguous int32 CUDA"):
            K._ints(bad, 3, "tok_off")
    assert K._ints(None, 3, "pos") is None
