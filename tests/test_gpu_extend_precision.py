"""How far the attention of query chunks is from 64 bits: the weights of the
values must not be held in so few bits that they show in a bf16 result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from shared_paged_kv_gb300 import kvs as K
from oracle import extend as OE
import harness as H
from test_gpu_extend import Batch, f64

DEV = H.DEV


def check(b, out, causal):
    """Every value within half a bf16 step of the output (2^-8 of it) and what
    the weights' two parts leave: the first part is the upper 16 bits of the
    float32 weight (less than 2^-7 of it remains), the second the remainder to
    half a bf16 step (2^-8): 2^-15 of sum p |V|.  The float32 share is that of
    assert_attention.  And the whole within the criterion of every attention
    of this library, 2e-3 (a bf16 rounding alone is 1.5e-3 to 1.7e-3)."""
    k, v = np.nan_to_num(f64(b.k), posinf=0.0), np.nan_to_num(f64(b.v), posinf=0.0)
    exp, mag, big = OE.extend_attention(f64(b.q), k, v, b.table, b.off, b.lens, 16, b.scale, causal)
    rows = ~np.isnan(exp[:, 0, 0])
    got, exp, mag = f64(out)[rows], exp[rows], mag[rows]
    eps = 2 * (b.d + 4) * 2.0 ** -24 * big + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(exp) + (2.0 ** -15 * (1 + 2.0 ** -8) + eps) * mag + 1e-30
    off = np.abs(got - exp)
    rel = np.linalg.norm(got - exp) / np.linalg.norm(exp)
    assert rel <= H.RTOL_L2, f"relative L2 {rel:.3e}"
    assert (off <= tol).all(), f"{(off > tol).sum()} of {off.size} off, most {(off / tol).max():.2f} of the tolerance"


@pytest.mark.parametrize("flags", [0, K.KVS_TEST_EXTEND_PLANNED])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 64), (16, 2, 128), (4, 4, 128), (10, 2, 128)])
@pytest.mark.parametrize("new, lens, prefix", [
    ([40, 7, 130], [700, 90, 333], 0),          # one launch, or pieces and their join
    ([3, 5, 2, 4], [1290, 1400, 1285, 1300], 1280),   # rows of all sequences over one prefix
    ([300], [300], 0),                          # a chunk from the start
])
def test_results_are_as_near_as_bf16_allows(new, lens, prefix, hq, hkv, d, causal, flags):
    b = Batch(new, lens, hq, hkv, d, prefix=prefix, seed=hq + d, pad=1, qscale=2.0)
    K.kvs_pool_set_test_flags(b.pool, flags)
    check(b, b.run(causal), causal)


@pytest.mark.parametrize("level", [2.0 ** -30, 2.0 ** -12, 2.0 ** 20])
def test_values_of_any_size(level):
    """The second part of a weight does not depend on the values' size, nor on
    how the sizes of different dimensions and blocks compare."""
    b = Batch([30, 2], [600, 500], 8, 2, 128, seed=11, qscale=2.0)
    b.v *= level
    b.v[..., ::3] *= 2.0 ** -20
    check(b, b.run(True), True)
    K.kvs_pool_set_test_flags(b.pool, 0)
    check(b, b.run(True), True)


@pytest.mark.parametrize("flags", [0, K.KVS_TEST_EXTEND_PLANNED])
def test_near_uniform_weights(flags):
    """Small queries: all weights lie within a few bf16 steps of one another."""
    b = Batch([20, 64], [900, 1000], 8, 2, 128, seed=12, qscale=2.0 ** -6)
    K.kvs_pool_set_test_flags(b.pool, flags)
    check(b, b.run(True), True)
