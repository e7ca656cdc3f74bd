"""Attention over a pool of microscaled 4-bit values without masses: no memory for scores is wanted."""
import numpy as np
import pytest
import torch

from oracle import mass as OM
from oracle import mx4 as O4
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace
from test_gpu_decode_mass import call, check, f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens, hq, hkv", [([700, 33], 8, 2), ([5000, 0, 2047], 12, 1), ([40] * 70, 4, 4)])
def test_the_smaller_workspace(lens, hq, hkv):
    s = make("mx4", lens, hq, hkv, 128, seed=hq)
    n = len(lens)
    size = K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MX4, n, s["mb"], hq)
    whole = K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MASS, n, s["mb"], hq)
    assert whole - size >= 4 * n * hq * s["mb"] * 64
    memory = workspace(size + 4096).fill_(0xC3)
    args = (s["pool"], 0, s["q"], hq, i32(s["table"]), s["mb"], i32(s["lens"]), n, s["scale"])
    out = torch.full((n, hq, 128), float("nan"), device=DEV)
    K.kvs_decode_attn_mx4(*args, out, memory[:size])
    assert (memory[size:] == 0xC3).all()
    want, _ = call(s, mass_in=None)
    assert torch.equal(out, want) and K.kvs_pool_check(s["pool"]) == 0
    with pytest.raises(K.KvsError):
        K.kvs_decode_attn_mx4(*args, out, memory[:size - 256])
    with pytest.raises(K.KvsError):     # with masses the scores are wanted
        K.kvs_decode_attn_mx4(*args, out, memory[:size], mass=torch.zeros_like(s["mass_in"]))
    wide = K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MX4, n, 2048, hq)
    assert wide == size                 # not a matter of the table's width


def test_of_pools_in_4_bits_alone():
    s = make("bf16", [20], 4, 2, 64)
    with pytest.raises(K.KvsError):
        K.kvs_workspace_size(s["pool"], K.KVS_OP_DECODE_MX4, 1, 2, 4)


@pytest.mark.parametrize("up", [100, 110])
def test_sums_of_large_values_stay_finite(up):
    """Values of up to 6 * 2^(1 + up): what they add up to over 2,000 tokens lies below 2^127, and so does every step."""
    s = make("mx4", [2000, 64, 700], 8, 2, 128, seed=up)
    s["scale"] /= 8                                  # weights of about one size
    for e in s["vsc"]:
        e[e < 255] += up
    s["values"][1] = s["values"][1] * 2.0 ** up
    out, mass = call(s)
    assert torch.isfinite(out).all()
    check(s, out, mass)


def test_warps_states_agree_on_their_references():
    """Sequences of two units, a warp each, whose tokens all have one score, values 1 in one and 0 in the other: the output
    is 1 / (1 + 2^(x1 - x0)).  The scores (base 2) lie between -64 and -32 and are exact products; what a warp's weights
    were taken against has to be what it is joined by, to the bit: half a last place at 64 is 2^-19, 1.3e-6 of a weight.
    Otherwise a warp's weights are off by 2^-22 (the exponential) and 2^-21 ln 2 (its argument, about 11, rounded): (1 - w) of
    twice 5.7e-7; the parts of a weight and their sum by 2^-23 each, the division by 2^-23, the factor of the join by 2^-22:
    1.2e-6 where 1 - w is at most 0.55."""
    n, hq = 60, 8
    s = make("mx4", [64] * n, hq, 1, 128, scales=(127, 128))
    kc, vc = s["k"][0], s["v"][0]
    kc.zero_(), vc.zero_()
    kc[..., 0] = 0x07                              # channel 0: 6, everywhere
    kc[:, :, 32:, 1] = 0x01                        # channel 2: 0.5 in the second half of a block
    vc[:, :, :32, :] = 0x22                        # values: 1 in the first half
    s["values"] = [np.where(np.isnan(x), 0, O4.dequantize(c.cpu().numpy(), np.full(x.shape[:3] + (4,), 127))) for x, c in zip(s["values"], (kc, vc))]
    q = np.zeros((n, hq, 128), np.float32)
    r = np.random.default_rng(0)
    q[..., 0] = -r.uniform(4.0, 7.0, (n, hq))      # 6 q log2(e) from -60 to -35
    q[..., 2] = r.uniform(-0.25, 0.25, (n, hq))    # half of it between the two scores
    s["q"], s["scale"] = torch.as_tensor(q).to(torch.bfloat16).to(DEV), 1.0
    out, mass = call(s, mass_in=None)
    want, _, w, _ = OM.attend(f64(s["q"]), *s["values"], s["table"], range(n + 1), s["lens"], 64, 1.0, False)
    assert 0.45 <= want.min() and want.max() <= 0.55
    assert np.abs(f64(out) / want - 1).max() <= 1.2e-6
