"""How many bits of a weight reach the values: decode attention with masses where nothing else is rounded much.

A query has one channel that is not 0, so a score is one product, exact in float32, and the exponential's argument is
rounded once: one of at most 8 (base 2) gives 8 * 2^-24 * ln 2 = 2^-21.5 of a weight at most, the exponential itself
2^-22.  Errors that differ from token to token, spread evenly below their limits, count in the norm of the output, whose
values are of either sign and independent of them, with 1 / sqrt(3): 2^-22.3 and 2^-22.8.  Of one sign they would count in
full, but in the row's sum as well, which takes them out again.  Sums: 2,048 tokens are at most 128 products of one warp, each added
with an error below 2^-24 of a partial sum, half of the whole on the mean: sqrt(128) * 2^-24 / sqrt(3) * 0.7 = 2^-21.8.
Together 2^-22.3 + 2^-22.8 + 2^-21.8 = 6e-7; the limit is 2^-20.3 = 7.7e-7.
Three bf16 parts keep all bits of a weight.  With two, emulated in 64 bits on such weights, the output is off by 1.8e-6 to
2.9e-6, so that a part cannot be lost unseen."""
import numpy as np
import pytest
import torch

from oracle import mass as OM

from test_gpu_decode_mass import call, f64, make

pytestmark = pytest.mark.gpu
LIMIT = 2.0 ** -20.3


def one_channel(s, seed, spread):
    r = np.random.default_rng(seed)
    q = np.zeros(s["q"].shape, np.float32)
    n, hq = q.shape[:2]
    at = r.integers(0, s["d"], (n, hq))
    size = r.uniform(0.3, 1.0, (n, hq)) * r.choice([-1, 1], (n, hq))
    q[np.arange(n)[:, None], np.arange(hq), at] = size
    s["q"] = torch.as_tensor(q).to(torch.bfloat16).cuda()
    # |k| stays below 5.5 (2.4 million normal values); the largest argument below 8
    s["scale"] = spread
    return s


@pytest.mark.parametrize("hq, hkv, d", [(8, 8, 128), (8, 2, 64), (16, 2, 128), (12, 1, 64), (16, 1, 128)])
def test_weights_over_bf16_pools_keep_their_bits(hq, hkv, d):
    s = one_channel(make("bf16", [2048, 777, 2040], hq, hkv, d, seed=d + hq), hq, 1.0)
    out, mass = call(s, mass_in=None)
    want, _, w, big = OM.attend(f64(s["q"]), s["values"][0], s["values"][1], s["table"], range(4), s["lens"], 16, s["scale"], False)
    assert big * 1.4427 <= 8
    for a in range(3):
        err = np.linalg.norm(f64(out)[a] - want[a]) / np.linalg.norm(want[a])
        assert err <= LIMIT, (a, err)


def test_weights_over_microscaled_pools():
    """The parts are fp16 there, at 2^11 and more of the largest weight: 2^-22 of a weight, and 2^-36 of the largest."""
    s = one_channel(make("mx4", [2048, 777, 2040], 8, 2, 128, seed=3, scales=(124, 127)), 5, 0.7)
    out, mass = call(s, mass_in=None)
    want, _, w, big = OM.attend(f64(s["q"]), s["values"][0], s["values"][1], s["table"], range(4), s["lens"], 64, s["scale"], False)
    assert big * 1.4427 <= 8
    for a in range(3):
        err = np.linalg.norm(f64(out)[a] - want[a]) / np.linalg.norm(want[a])
        assert err <= LIMIT, (a, err)
