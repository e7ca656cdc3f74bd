"""Pins of the oracle's weights by token and of its 4-bit floating point."""
import numpy as np
import pytest

from oracle import extend as OE
from oracle import mass as OM
from oracle import mx4 as O4


def test_scale_and_codes_by_hand():
    x = np.zeros(32)
    x[:8] = [7.0, -6.0, 5.0, 2.5, 0.25, -0.75, 1.75, 3.5]     # 4 <= 7 < 8: scale 1
    codes, e = O4.quantize(x)
    assert e.tolist() == [127]
    assert O4.dequantize(codes, e)[:8].tolist() == [6.0, -6.0, 4.0, 2.0, 0.0, -1.0, 2.0, 4.0]
    assert codes[0] == 0x7 | (0xF << 4)
    codes, e = O4.quantize(np.ldexp(x, 10))
    assert e.tolist() == [137] and O4.dequantize(codes, e)[2] == 4096
    codes, e = O4.quantize(np.zeros(64))
    assert e.tolist() == [0, 0] and not codes.any()
    assert O4.quantize(np.full(32, 2.0 ** -130))[1].tolist() == [0]


def test_values_that_are_held_come_back():
    r = np.random.default_rng(0)
    codes = r.integers(0, 256, (50, 64)).astype(np.uint8)
    codes[:, ::16] = 0x66                                       # a 4 in every group: the scale is the held one
    scales = r.integers(5, 250, (50, 4)).astype(np.uint8)
    x = O4.dequantize(codes, scales)
    c2, s2 = O4.quantize(x)
    assert (s2 == scales).all() and (O4.dequantize(c2, s2) == x).all()


def test_error_is_half_a_step():
    x = np.random.default_rng(1).standard_normal((100, 64))
    c, s = O4.quantize(x)
    step = np.exp2(s.astype(float) - 127).repeat(32, -1)
    y = O4.dequantize(c, s)
    gap = np.where(np.abs(x) / step < 2, 0.25, np.where(np.abs(x) / step < 4, 0.5, 1.0)) * step
    clipped = np.abs(x) > 6 * step
    assert (np.abs(y - x)[~clipped] <= gap[~clipped]).all() and (np.abs(y)[clipped] == 6 * step[clipped]).all()


@pytest.mark.parametrize("causal", [True, False])
def test_weights_against_the_attention_oracle(causal):
    r = np.random.default_rng(2)
    hq, hkv, d, lens, off = 4, 2, 8, [21, 5, 0], [0, 3, 5, 5]
    k, v = r.standard_normal((6, hkv, 16, d)), r.standard_normal((6, hkv, 16, d))
    table = np.array([[3, 1], [0, -1], [-1, -1]])
    q = r.standard_normal((5, hq, d))
    out, _, mass, _ = OM.attend(q, k, v, table, off, lens, 16, 0.5, causal)
    np.testing.assert_allclose(out, OE.extend_attention(q, k, v, table, off, lens, 16, 0.5, causal)[0], rtol=1e-12)
    assert [len(m) for m in mass] == lens
    np.testing.assert_allclose([m.sum() for m in mass], [3 * hq, 2 * hq, 0], rtol=1e-12)   # a row's weights add up to 1


def test_a_bad_block_takes_its_tokens_out():
    k = np.ones((2, 1, 16, 4))
    _, _, mass, _ = OM.attend(np.ones((1, 1, 4)), k, k, [[0, 9, 1]], [0, 1], [40], 16, 1.0, False)
    np.testing.assert_allclose(mass[0], np.r_[np.full(16, 1 / 24), np.zeros(16), np.full(8, 1 / 24)])
