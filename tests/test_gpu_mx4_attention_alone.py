"""Attention over a pool of microscaled 4-bit values without masses: no memory for scores is wanted."""
import pytest
import torch

from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace
from test_gpu_decode_mass import call, check, make

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
