"""Cases of the operators that make room in a shared paged KV pool: decode attention that adds up the attention weight
of every stored token, the same weights of a chunk of query rows, the choice of the tokens worth keeping with the
compaction of their blocks, and a pool of microscaled 4-bit floating-point values (append, read-back, decode attention).

`run` computes each either in elementary torch operations (own = False) or by the library's calls (own = True).
Sequence a holds seq_len[a] tokens in the blocks of its table row; mass[a][t] is the attention weight that token t
has gathered, over all query heads and rows.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"bf16": 16, "mx4": 64}
MX_GROUP = 32                                     # values that share one power-of-two scale
MX_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- cases ----
def listed():
    return [
        # one decode step of four small agents: launches and their chains count
        {"name": "mass_step_small", "op": "decode", "pool": "bf16", "mass": True, "n_seq": 4, "hq": 8, "hkv": 2, "d": 64,
         "prefix": 0, "ctx_lo": 300, "ctx_hi": 384, "mix": 1},
        # one decode step of 32 agents with one system prompt, eight query heads to a KV head
        {"name": "mass_step_fanout", "op": "decode", "pool": "bf16", "mass": True, "n_seq": 32, "hq": 16, "hkv": 2, "d": 128,
         "prefix": 4096, "ctx_lo": 512, "ctx_hi": 2048, "mix": 2},
        # one decode step of eight long-running agents, every head with its own keys
        {"name": "mass_step_mha", "op": "decode", "pool": "bf16", "mass": True, "n_seq": 8, "hq": 32, "hkv": 32, "d": 128,
         "prefix": 0, "ctx_lo": 9830, "ctx_hi": 16384, "mix": 3},
        # which prompt tokens the last rows of eight prompts look at, before the prompts are thinned out
        {"name": "chunk_mass_window", "op": "chunk", "n_seq": 8, "hq": 32, "hkv": 8, "d": 128, "new_lo": 32, "new_hi": 32,
         "ctx_lo": 3500, "ctx_hi": 8192, "causal": True, "mix": 4},
        # the weights of all rows of a long prompt
        {"name": "chunk_mass_prompt", "op": "chunk", "n_seq": 1, "hq": 32, "hkv": 8, "d": 128, "new_lo": 8192,
         "new_hi": 8192, "ctx_lo": 0, "ctx_hi": 0, "causal": True, "mix": 5},
        # four small agents fork from their histories and keep a third of them
        {"name": "evict_small", "op": "evict", "pool": "bf16", "n_seq": 4, "hkv": 2, "d": 64, "layers": 1, "ctx_lo": 300,
         "ctx_hi": 384, "budget": 128, "first": 4, "recent": 32, "mix": 6},
        # 32 agents fork from one another's histories and keep 2,048 tokens each
        {"name": "evict_agents", "op": "evict", "pool": "bf16", "n_seq": 32, "hkv": 2, "d": 128, "layers": 4, "ctx_lo": 4608,
         "ctx_hi": 6144, "budget": 2048, "first": 16, "recent": 256, "mix": 7},
        # one very long history in 4 bits loses three quarters of its tokens
        {"name": "evict_long_mx4", "op": "evict", "pool": "mx4", "n_seq": 1, "hkv": 8, "d": 128, "layers": 8,
         "ctx_lo": 131072, "ctx_hi": 131072, "budget": 32768, "first": 64, "recent": 4096, "mix": 8},
        # one decode step of 12 agents appends to a 4-bit cache
        {"name": "append_step_mx4", "op": "append", "n_seq": 12, "hq": 32, "hkv": 8, "new_lo": 1, "new_hi": 1,
         "ctx_lo": 4000, "ctx_hi": 8191, "axes": 1, "theta": 1e6, "mix": 9},
        # ragged prompts of 12 agents, appended and read back
        {"name": "append_prompts_mx4", "op": "append", "n_seq": 12, "hq": 32, "hkv": 8, "new_lo": 257, "new_hi": 1023,
         "ctx_lo": 0, "ctx_hi": 4000, "axes": 1, "theta": 1e6, "mix": 10},
        # one decode step of 12 agents over a 4-bit cache
        {"name": "decode_step_mx4", "op": "decode", "pool": "mx4", "mass": False, "n_seq": 12, "hq": 32, "hkv": 8, "d": 128,
         "prefix": 0, "ctx_lo": 4000, "ctx_hi": 8191, "mix": 11},
        # eight agents with long histories in 4 bits, their weights added up
        {"name": "decode_mass_long_mx4", "op": "decode", "pool": "mx4", "mass": True, "n_seq": 8, "hq": 32, "hkv": 8,
         "d": 128, "prefix": 0, "ctx_lo": 16384, "ctx_hi": 32768, "mix": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    """What a case's plain form takes, in padded values or scores."""
    if c["op"] == "decode":
        return c["n_seq"] * c["hkv"] * c["d"] * (c["prefix"] + c["ctx_hi"])
    if c["op"] == "chunk":
        return c["n_seq"] * c["hq"] * c["new_hi"] * (c["new_hi"] + c["ctx_hi"])
    if c["op"] == "evict":
        return c["n_seq"] * c["hkv"] * c["d"] * c["layers"] * c["ctx_hi"]
    return c["n_seq"] * c["hkv"] * c["new_hi"]


def draw(rng):
    while True:
        op = rng.choice(["decode", "decode", "decode", "chunk", "chunk", "evict", "evict", "append"])
        hq, hkv = rng.choice([(16, 2), (32, 32), (32, 8), (8, 2), (8, 8), (20, 4), (40, 8), (12, 1), (16, 1)])
        c = {"op": op, "n_seq": _log(rng, 1, 64), "hkv": hkv, "mix": rng.randrange(1, 1 << 30)}
        if op == "decode":
            pool = rng.choice(["bf16", "bf16", "mx4"])
            hi = _log(rng, 1, 32768)
            c.update(pool=pool, mass=pool == "bf16" or rng.random() < 0.5, hq=hq, d=128 if pool == "mx4" else rng.choice([64, 128]),
                     prefix=64 * rng.choice([0, 0, rng.randint(0, 64)]), ctx_lo=rng.randint(1, hi), ctx_hi=hi)
        elif op == "chunk":
            hi = _log(rng, 1, 8192)
            c.update(hq=hq, d=rng.choice([64, 128]), new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0,
                     ctx_hi=_log(rng, 1, 16384), causal=rng.random() < 0.8)
        elif op == "evict":
            pool = rng.choice(["bf16", "bf16", "mx4"])
            hi = _log(rng, 2, 131072)
            c.update(pool=pool, d=128 if pool == "mx4" else rng.choice([64, 128]), layers=rng.randint(1, 8),
                     ctx_lo=rng.randint(1, hi), ctx_hi=hi, budget=rng.randint(0, hi), first=rng.randint(0, 64),
                     recent=_log(rng, 1, 4096))
        else:
            hi = _log(rng, 1, 1023)
            c.update(n_seq=_log(rng, 1, 12 if hi > 100 else 64), hq=hq, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0,
                     ctx_hi=rng.randint(0, 60000), axes=rng.choice([0, 1]), theta=rng.choice([1e4, 1e6]))
        if _cost(c) <= max(_cost(x) for x in listed() if x["op"] == op):
            return c


def _lens(c):
    """(new tokens, tokens before them) of every sequence."""
    r = np.random.RandomState(c["mix"] % (1 << 31))
    new = r.randint(c["new_lo"], c["new_hi"] + 1, c["n_seq"]) if "new_lo" in c else np.zeros(c["n_seq"], np.int64)
    return new, r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["n_seq"])


# -------------------------------------------------------------- inputs ----
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


def _slab(gen, pool, cap, hkv, block, d):
    """(values or codes, scales or None) of one layer's keys or values: heads and channels of unequal size."""
    size = torch.exp2(torch.randn(hkv, 1, d, generator=gen, device="cuda") * 0.5)
    x = (torch.randn(cap, hkv, block, d, generator=gen, device="cuda") * size).to(torch.bfloat16)
    if pool == "bf16":
        return x, None
    code, scale = torch.empty(cap, hkv, block, d // 2, dtype=torch.uint8, device="cuda"), None
    scale = torch.empty(cap, hkv, block, d // MX_GROUP, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * block * d))
    for b in range(0, cap, step):
        code[b:b + step], scale[b:b + step], _ = _quantise(x[b:b + step])
    return code, scale


def _fill_pool(s, gen, c, cap, layers, n):
    block = BLOCK[c["pool"]]
    ks = [_slab(gen, c["pool"], cap, c["hkv"], block, c["d"]) for _ in range(layers)]
    vs = [_slab(gen, c["pool"], cap, c["hkv"], block, c["d"]) for _ in range(layers)]
    s.update(k=[x for x, _ in ks], v=[x for x, _ in vs], ksc=[x for _, x in ks], vsc=[x for _, x in vs], block=block)
    if own:
        from shared_paged_kv_gb300 import kvs as K
        mx = c["pool"] == "mx4"
        s["handle"] = K.kvs_pool_create(layers, c["hkv"], c["d"], block, K.KVS_DTYPE_MX4 if mx else K.KVS_DTYPE_BF16, cap, n,
                                        s["k"], s["v"], s["ksc"] if mx else None, s["vsc"] if mx else None)


def _table(rng, n, prefix_blocks, blocks, spare=0):
    """Shuffled blocks: `prefix_blocks` common ones, then own ones, `blocks` in all for each sequence."""
    rest = np.maximum(blocks - prefix_blocks, 0)
    cap = max(1, int(prefix_blocks + rest.sum()) + spare)
    ids = rng.permutation(cap)
    table = np.full((n, max(1, int(blocks.max()))), -1)
    k = prefix_blocks
    for a in range(n):
        table[a, :prefix_blocks] = ids[:prefix_blocks]
        table[a, prefix_blocks:prefix_blocks + rest[a]] = ids[k:k + rest[a]]
        k += rest[a]
    return table, cap, ids[k:]


def _gathered(gen, n, width, level, spread=1.0):
    """Weights as a history of steps leaves them: few heavy tokens, many light ones, some never looked at."""
    x = level * torch.exp(spread * torch.randn(n, width, generator=gen, device="cuda"))
    return torch.where(torch.rand(n, width, generator=gen, device="cuda") < 0.05, 0.0, x)


def prepare(case, seed):
    c = case
    gen, rng = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n, (new, ctx) = c["n_seq"], _lens(c)
    s = {"case": c}
    if c["op"] == "decode":
        lens = c["prefix"] + ctx
        block = BLOCK[c["pool"]]
        table, cap, _ = _table(rng, n, c["prefix"] // block, -(-lens // block))
        _fill_pool(s, gen, c, cap, 1, n)
        mb = table.shape[1]
        s.update(table=_i32(table), seq_len=_i32(lens), max_blocks=mb, longest=int(lens.max()),
                 q=1.5 * _randn(gen, n, c["hq"], c["d"]), mass_in=_gathered(gen, n, mb * block, c["hq"] / max(1.0, lens.mean())),
                 out=torch.empty(n, c["hq"], c["d"], device="cuda"))
        s["mass"] = s["mass_in"].clone()
        if own:
            from shared_paged_kv_gb300 import kvs as K
            s["ws"] = torch.empty(K.kvs_workspace_size(s["handle"], K.KVS_OP_DECODE_MASS, n, mb, c["hq"]), dtype=torch.uint8,
                                  device="cuda")
    elif c["op"] == "chunk":
        lens = ctx + (new if c["causal"] else 1)
        table, cap, _ = _table(rng, n, 0, -(-lens // BLOCK["bf16"]))
        _fill_pool(s, gen, dict(c, pool="bf16"), cap, 1, n)
        mb, total = table.shape[1], int(new.sum())
        s.update(table=_i32(table), seq_len=_i32(lens), max_blocks=mb, longest=int(lens.max()), most_new=int(new.max()),
                 tok_off=_i32(np.concatenate([[0], np.cumsum(new)])), tokens=total,
                 q=1.5 * _randn(gen, total, c["hq"], c["d"]), mass_in=_gathered(gen, n, mb * s["block"], c["hq"] * total / max(1, lens.sum())))
        s["mass"] = s["mass_in"].clone()
        if own:
            from shared_paged_kv_gb300 import kvs as K
            s["ws"] = torch.empty(K.kvs_extend_mass_workspace_size(s["handle"], total, n, mb, c["hq"]), dtype=torch.uint8,
                                  device="cuda")
    elif c["op"] == "evict":
        # every sequence is a fork: its blocks are also referenced by the history that it came from, which goes on
        block = BLOCK[c["pool"]]
        blocks = -(-ctx // block)
        spare = int((-(-np.minimum(ctx, np.maximum(c["budget"], c["first"] + c["recent"])) // block)).sum()) + 3
        table, cap, free = _table(rng, n, 0, blocks, spare)
        _fill_pool(s, gen, c, cap, c["layers"], n)
        mb = table.shape[1]
        refs = np.zeros(cap, np.int64)
        for a in range(n):
            refs[table[a, :blocks[a]]] = 2
        parts = [("table", table.ravel()), ("seq_len", ctx), ("refcount", refs),
                 ("free_ids", np.concatenate([np.sort(free)[::-1], np.zeros(cap - len(free))])), ("n_free", [len(free)])]
        sizes = [(name, len(x)) for name, x in parts]
        sizes.append(("mass", n * mb * block))
        # what a pass changes lies in one buffer, so that a pass can begin again from `before`
        pad = [-(-k // 4) * 4 for _, k in sizes]
        before = torch.zeros(sum(pad), dtype=torch.int32, device="cuda")
        now, at = torch.empty_like(before), 0
        for (name, k), p in zip(sizes, pad):
            s[name] = now[at:at + k]
            if name == "mass":
                s[name] = s[name].view(torch.float32).view(n, mb * block)
                before[at:at + k] = _gathered(gen, n, mb * block, 1e-2, 2.5).view(torch.int32).flatten()
            else:
                before[at:at + k] = _i32(dict(parts)[name])
            at += p
        s["table"] = s["table"].view(n, mb)
        most = int(np.minimum(ctx, np.maximum(c["budget"], c["first"] + c["recent"])).sum())
        s.update(before=before, now=now, max_blocks=mb, longest=int(ctx.max()), kept=most,
                 budget=torch.full((n,), c["budget"], dtype=torch.int32, device="cuda"),
                 idx=torch.zeros(most, dtype=torch.int32, device="cuda"),
                 idx_off=torch.zeros(n + 1, dtype=torch.int64, device="cuda"))
        if own:
            from shared_paged_kv_gb300 import kvs as K
            s["ws"] = torch.empty(K.kvs_workspace_size(s["handle"], K.KVS_OP_COMPACT, n, mb), dtype=torch.uint8, device="cuda")
    else:
        block, d = BLOCK["mx4"], 128
        lens = ctx + new
        mb = max(1, int(-(-lens.max() // block)))
        lo, hi = ctx // block, -(-lens // block)                      # blocks that new tokens go to
        n_new = int((hi - lo).sum())
        cap = n_new + max(4, n_new // 8)
        ids = rng.permutation(cap)
        table = ids[n_new + rng.randint(0, cap - n_new, (n, mb))]     # the history's blocks, not touched
        k = 0
        for a in range(n):
            table[a, lo[a]:hi[a]] = ids[k:k + hi[a] - lo[a]]
            k += hi[a] - lo[a]
        _fill_pool(s, gen, dict(c, pool="mx4", d=d), cap, 1, n)
        total = int(new.sum())
        s.update(table=_i32(table), seq_len=_i32(lens), max_blocks=mb, tok_off=_i32(np.concatenate([[0], np.cumsum(new)])),
                 tokens=total, k_new=_randn(gen, total, c["hkv"], d), v_new=_randn(gen, total, c["hkv"], d),
                 q=_randn(gen, total, c["hq"], d))
        s.update(k_rows=torch.empty_like(s["k_new"]), v_rows=torch.empty_like(s["v_new"]), q_out=torch.empty_like(s["q"]))
        if own:
            from shared_paged_kv_gb300 import kvs as K
            s["rope"] = K.RopeAxes(c["theta"], (d // 2,)) if c["axes"] else None
    return s


# ----------------------------------------------------------------- run ----
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from shared_paged_kv_gb300 import kvs as K
    c = s["case"]
    n, mb = c["n_seq"], s["max_blocks"]
    if c["op"] == "decode":
        scale = 1.0 / math.sqrt(c["d"])
        if c["pool"] == "mx4":
            K.kvs_decode_attn_mx4(s["handle"], 0, s["q"], c["hq"], s["table"], mb, s["seq_len"], n, scale, s["out"], s["ws"],
                                  mass_in=s["mass_in"] if c["mass"] else None, carry=0.75,
                                  mass=s["mass"] if c["mass"] else None)
        else:
            K.kvs_decode_attn_mass(s["handle"], 0, s["q"], c["hq"], s["table"], mb, s["seq_len"], n, scale, s["out"],
                                   s["mass_in"], 0.75, s["mass"], s["ws"])
        return (s["out"], s["mass"]) if c["mass"] else s["out"]
    if c["op"] == "chunk":
        K.kvs_extend_mass(s["handle"], 0, s["q"], s["tokens"], s["tok_off"], c["hq"], s["table"], mb, s["seq_len"], n,
                          c["causal"], 1.0 / math.sqrt(c["d"]), s["mass_in"], 0.75, s["mass"], s["ws"])
        return s["mass"]
    if c["op"] == "evict":
        s["now"].copy_(s["before"])
        K.kvs_keep_heavy(s["handle"], s["mass"], s["seq_len"], n, mb, s["budget"], c["first"], c["recent"], s["idx"],
                         s["idx_off"])
        K.kvs_compact(s["handle"], s["table"], mb, s["seq_len"], n, s["idx"], s["idx_off"], s["refcount"], s["free_ids"],
                      s["n_free"], s["ws"], mass=s["mass"])
        return _evict_outputs(s)
    K.kvs_append(s["handle"], 0, s["k_new"], s["v_new"], s["tokens"], s["tok_off"], s["table"], mb, s["seq_len"], n,
                 rope=s["rope"], q=s["q"], n_q_heads=c["hq"], q_out=s["q_out"])
    K.kvs_gather(s["handle"], 0, s["tokens"], s["tok_off"], s["table"], mb, s["seq_len"], n, s["k_rows"], s["v_rows"])
    return s["k_rows"], s["v_rows"], s["q_out"]


def _evict_outputs(s):
    """Kept tokens, the sequences' new state, and the pool."""
    return {"idx": s["idx"], "idx_off": s["idx_off"], "table": s["table"], "seq_len": s["seq_len"], "refcount": s["refcount"],
            "n_free": s["n_free"], "mass": s["mass"], "k": s["k"], "v": s["v"], "ksc": s["ksc"], "vsc": s["vsc"]}


def _quantise(x):
    """Codes (two to a byte, the first in the low four bits), scale bytes, and the values they stand for: a group's scale
    is the power of two that puts its largest magnitude between 4 and 8, a value the nearest of MX_VALUES, ties to even."""
    g = x.to(torch.bfloat16).float().unflatten(-1, (-1, MX_GROUP))
    top = torch.frexp(g.abs().amax(-1))
    scale = torch.where(top.mantissa > 0, top.exponent - 3 + 127, 0).clamp(0, 254).to(torch.int32)
    y = torch.ldexp(g, 127 - scale[..., None]).double().abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0).float()
    code = torch.bucketize(y, torch.tensor(MX_VALUES, device=x.device)).to(torch.uint8)
    sign = torch.signbit(g)
    value = torch.ldexp(torch.where(sign, -y, y), scale[..., None] - 127).flatten(-2)
    code = (code | (sign.to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.uint8), value


def _values(code, scale):
    """What codes and scale bytes stand for, in 32 bits."""
    lut = torch.tensor(MX_VALUES + [-v for v in MX_VALUES], device=code.device)
    x = torch.stack([lut[(code & 15).long()], lut[(code >> 4).long()]], -1).flatten(-2)
    return torch.ldexp(x.unflatten(-1, (-1, MX_GROUP)), scale[..., None].to(torch.int32) - 127).flatten(-2)


def _dense(s, slab, scale, length):
    """One layer's rows of every sequence, [n][hkv][length][d] in 32 bits; rows behind a sequence's end are zeros."""
    ids = s["table"].long().clamp(min=0)
    x = slab[ids].float() if scale is None else _values(slab[ids], scale[ids])
    x = x.transpose(2, 3).flatten(1, 2)[:, :length].transpose(1, 2)
    seen = torch.arange(length, device=x.device) < s["seq_len"].long()[:, None]
    return torch.where(seen[:, None, :, None], x, 0.0)


def _add_mass(s, weights, length):
    """carry * mass_in + weights over the stored tokens; the others stay as they were."""
    seen = torch.arange(length, device=weights.device) < s["seq_len"].long()[:, None]
    m = s["mass_in"][:, :length]
    s["mass"][:, :length] = torch.where(seen, 0.75 * m + weights, m)
    return s["mass"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "decode":
        n, hq, hkv, d, L = c["n_seq"], c["hq"], c["hkv"], c["d"], s["longest"]
        q = s["q"].float().view(n, hkv, hq // hkv, d)
        w = q @ _dense(s, s["k"][0], s["ksc"][0], L).transpose(2, 3)
        w *= 1.0 / math.sqrt(d)
        hidden = torch.arange(L, device="cuda") >= s["seq_len"].long()[:, None]
        w.masked_fill_(hidden[:, None, None], -math.inf)
        w -= w.amax(-1, keepdim=True)
        w.exp_()
        w /= w.sum(-1, keepdim=True)
        out = (w @ _dense(s, s["v"][0], s["vsc"][0], L)).view(n, hq, d)
        return (out, _add_mass(s, w.sum((1, 2)), L)) if c["mass"] else out
    if c["op"] == "chunk":
        return _add_mass(s, _chunk_weights(s), s["longest"])
    if c["op"] == "evict":
        s["now"].copy_(s["before"])
        return _evict_plain(s)
    k, q = s["k_new"].float(), s["q"].float()
    off, lens = s["tok_off"].long(), s["seq_len"].long()
    seq = torch.repeat_interleave(torch.arange(c["n_seq"], device="cuda"), off[1:] - off[:-1], output_size=s["tokens"])
    place = lens[seq] - off[seq + 1] + torch.arange(s["tokens"], device="cuda")
    if c["axes"]:
        w = c["theta"] ** (-2.0 * torch.arange(64, dtype=torch.float64, device="cuda") / 128)
        ang = (place.double()[:, None] * w)[:, None]
        cs, sn = ang.cos().float(), ang.sin().float()
        k, q = _turn(k, cs, sn), _turn(q, cs, sn)
    blk, at = s["table"].long()[seq, place // s["block"]], place % s["block"]
    kc, ks, kv = _quantise(k)
    vc, vs, vv = _quantise(s["v_new"])
    s["k"][0][blk, :, at], s["ksc"][0][blk, :, at] = kc, ks
    s["v"][0][blk, :, at], s["vsc"][0][blk, :, at] = vc, vs
    return kv.to(torch.bfloat16), vv.to(torch.bfloat16), q.to(torch.bfloat16)


def _turn(x, cs, sn):
    lo, hi = x[..., :64], x[..., 64:]
    return torch.cat([lo * cs - hi * sn, hi * cs + lo * sn], dim=-1)


def _chunk_weights(s):
    """[n][longest]: the attention weights of a sequence's rows, summed over rows and heads."""
    c = s["case"]
    n, hq, hkv, d, L, Q = c["n_seq"], c["hq"], c["hkv"], c["d"], s["longest"], s["most_new"]
    g = hq // hkv
    off, lens = s["tok_off"].long(), s["seq_len"].long()
    j = torch.arange(Q, device="cuda")
    live = j < (off[1:] - off[:-1])[:, None]                                          # [n][Q]
    q = torch.where(live[..., None, None], s["q"][(off[:-1, None] + j).clamp(max=s["tokens"] - 1)].float(), 0.0)
    lim = (lens - (off[1:] - off[:-1]))[:, None] + j + 1 if c["causal"] else lens[:, None].expand(n, Q)
    lim = torch.where(live, torch.minimum(lim, lens[:, None]), 0)
    w = q.view(n, Q, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, Q * g, d) @ _dense(s, s["k"][0], None, L).transpose(2, 3)
    w *= 1.0 / math.sqrt(d)
    w.masked_fill_(torch.arange(L, device="cuda") >= lim.repeat_interleave(g, 1)[:, None, :, None], -math.inf)
    w -= w.amax(-1, keepdim=True).clamp(min=-1e30)
    w.exp_()
    w /= w.sum(-1, keepdim=True).clamp(min=1e-30)
    return w.sum((1, 2))


def _evict_plain(s):
    c, block = s["case"], s["block"]
    n, L, mb, dev = c["n_seq"], s["longest"], s["max_blocks"], s["mass"].device
    lens, t = s["seq_len"].long(), torch.arange(L, device=dev)
    stored = t < lens[:, None]
    must = stored & ((t < c["first"]) | (t >= (lens - c["recent"])[:, None]))
    count = torch.maximum(must.sum(1), torch.minimum(lens, s["budget"].long()))
    m = torch.where(must, math.inf, torch.where(stored, s["mass"][:, :L], -math.inf))
    order = torch.argsort(m, dim=1, descending=True, stable=True)
    keep = torch.zeros(n, L, dtype=torch.bool, device=dev).scatter_(1, order, t < count[:, None])
    seq, idx = keep.nonzero(as_tuple=True)                            # ascending within each sequence
    off = torch.cat([count.new_zeros(1), count.cumsum(0)])
    s["idx_off"].copy_(off)
    s["idx"][:idx.numel()] = idx
    to = torch.arange(idx.numel(), device=dev) - off[seq]
    # blocks from the first one whose rows change on are written: those that others reference are replaced
    b = torch.arange(mb, device=dev)
    old, new = (lens + block - 1) // block, (count + block - 1) // block
    same = keep.long().cumprod(1).sum(1)
    first = torch.where(same >= count, new, same // block)
    table, held = s["table"].long(), b < old[:, None]
    refs = s["refcount"].long()
    written = (b >= first[:, None]) & (b < new[:, None])
    fresh = written & (refs[table.clamp(min=0)] > 1)
    gone = held & (b >= new[:, None])
    free = s["n_free"].long()
    took = torch.cumsum(fresh.flatten().long(), 0).view(n, mb)
    ids = torch.where(fresh, s["free_ids"].long()[(free - took).clamp(min=0)], table)
    left = refs.scatter_add(0, table.clamp(min=0).flatten(), -(fresh | gone).flatten().long())
    left[ids[fresh]] = 1
    for layer in range(c["layers"]):
        for slab in (s["k"][layer], s["v"][layer], s["ksc"][layer], s["vsc"][layer]):
            if slab is not None:
                slab[ids[seq, to // block], :, to % block] = slab[table[seq, idx // block], :, idx % block]
    back = ((refs > 0) & (left == 0)).nonzero().flatten().flip(0)
    rest = free - took.flatten()[-1:]
    s["free_ids"][rest + torch.arange(back.numel(), device=dev)] = back.to(torch.int32)
    s["n_free"].copy_(rest + back.numel())
    s["refcount"].copy_(left)
    s["table"].copy_(torch.where(gone, -1, ids))
    moved = s["mass"][seq, idx]
    s["mass"][:, :L] = torch.where(stored, 0.0, s["mass"][:, :L])
    s["mass"][seq, to] = moved
    s["seq_len"].copy_(count)
    return _evict_outputs(s)


# ---------------------------------------------------------------- work ----
def _row_bytes(pool, d):
    return 2 * d if pool == "bf16" else d // 2 + d // MX_GROUP


def work(case):
    c = case
    new, ctx = _lens(c)
    n, hkv = c["n_seq"], c["hkv"]
    if c["op"] == "decode":
        lens = c["prefix"] + ctx
        unique, every = c["prefix"] + int(ctx.sum()), int(lens.sum())
        b = 2 * unique * hkv * _row_bytes(c["pool"], c["d"]) + n * c["hq"] * c["d"] * (2 + 4) + (8 * every if c["mass"] else 0)
        return {"bytes": b, "flops": 4 * c["d"] * c["hq"] * every}
    if c["op"] == "chunk":
        lens, t = ctx + (new if c["causal"] else 1), int(new.sum())
        seen = sum((m * (x - m) + m * (m + 1) // 2) if c["causal"] else m * x for m, x in zip(new.tolist(), lens.tolist()))
        return {"bytes": int(lens.sum()) * (hkv * c["d"] * 2 + 8) + t * c["hq"] * c["d"] * 2, "flops": 2 * c["d"] * c["hq"] * seen}
    if c["op"] == "evict":
        kept = int(np.minimum(ctx, np.maximum(c["budget"], c["first"] + c["recent"])).sum())
        rows = 2 * 2 * kept * hkv * _row_bytes(c["pool"], c["d"]) * c["layers"]
        return {"bytes": rows + 4 * int(ctx.sum()) + 4 * kept, "flops": int(ctx.sum())}
    t, row = int(new.sum()), 2 * hkv * 128 * 2
    return {"bytes": t * (2 * row + 2 * 2 * hkv * _row_bytes("mx4", 128) + 2 * c["hq"] * 128 * 2),
            "flops": t * 128 * (3 * (c["hq"] + hkv) + 2 * 6 * hkv)}


# --------------------------------------------------------------- exact ----
def _exact_rows(s, which, a, h, length):
    """One head's rows of sequence a in 64 bits."""
    ids = s["table"][a, : -(-length // s["block"])].long()
    x = s[which][0][ids, h]
    if x.dtype != torch.uint8:
        return x.reshape(-1, x.shape[-1])[:length].double()
    nib = torch.stack([x & 15, x >> 4], -1).reshape(-1, x.shape[-1] * 2)[:length].long()
    e, m = (nib >> 1) & 3, (nib & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m)) * (1 - 2 * (nib >> 3).double())
    sc = s[which + "sc"][0][ids, h].reshape(-1, v.shape[-1] // MX_GROUP)[:length].double() - 127
    return v * torch.exp2(sc).repeat_interleave(MX_GROUP, 1)


def _exact_held(x):
    """The nearest 4-bit values of bf16 rows under their groups' scales, by distance to each of the sixteen."""
    g = x.to(torch.bfloat16).double().unflatten(-1, (-1, MX_GROUP))
    top = g.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 2).clamp(min=2.0 ** -127)
    even = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=x.device)  # first on a tie
    pick = torch.stack([(g.abs() / scale - v).abs() for v in even], -1).argmin(-1)
    return (even[pick] * torch.sign(g) * scale).flatten(-2)


def exact(case, seed):
    c = case
    if c["op"] == "chunk" and 2.0 * c["d"] * _cost(c) > 4e12:
        return None
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    n, hkv = c["n_seq"], c["hkv"]
    if c["op"] in ("decode", "chunk"):
        hq, d = c["hq"], c["d"]
        g, lens = hq // hkv, s["seq_len"].tolist()
        off = s["tok_off"].tolist() if c["op"] == "chunk" else list(range(n + 1))
        mass = s["mass_in"].double()
        out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
        for a in range(n):
            m, x = off[a + 1] - off[a], lens[a]
            mass[a, :x] *= 0.75
            for h in range(hkv):
                K = _exact_rows(s, "k", a, h, x)
                V = _exact_rows(s, "v", a, h, x) if c["op"] == "decode" else None
                for e in range(h * g, h * g + g):
                    S = s["q"][off[a]:off[a + 1], e].double() @ K.T / math.sqrt(d)
                    if c["op"] == "chunk" and c["causal"]:
                        S.masked_fill_(torch.ones_like(S, dtype=torch.bool).triu(x - m + 1), -math.inf)
                    S = torch.softmax(S, -1)
                    mass[a, :x] += S.sum(0)
                    if V is not None:
                        out[a, e] = S[0] @ V
        return mass if c["op"] == "chunk" else (out, mass) if c["mass"] else out
    if c["op"] == "append":
        off, lens = s["tok_off"].tolist(), s["seq_len"].tolist()
        k, q = s["k_new"].double(), s["q"].double()
        if c["axes"]:
            pos = torch.cat([torch.arange(lens[a] - off[a + 1] + off[a], lens[a], device="cuda") for a in range(n)]).double()
            ang = pos[:, None] * (float(c["theta"]) ** (-torch.arange(64, device="cuda").double() / 64))
            z = torch.polar(torch.ones_like(ang), ang)[:, None]
            turn = lambda x: torch.view_as_real(torch.complex(x[..., :64], x[..., 64:]) * z).transpose(-1, -2).flatten(-2)  # noqa: E731
            k, q = turn(k), turn(q)
        return _exact_held(k), _exact_held(s["v_new"]), q
    # eviction, one sequence after the other on the host; rows of the pool are copied, so they stay as they are
    s["now"].copy_(s["before"])
    block, lens = s["block"], s["seq_len"].tolist()
    mass, table, refs = s["mass"].double().cpu().numpy(), s["table"].cpu().numpy(), s["refcount"].cpu().numpy()
    free = s["free_ids"][: int(s["n_free"])].tolist()
    start = refs.copy()
    lists, moves, gone = [], [], []
    for a in range(n):
        x = lens[a]
        must = [t for t in range(x) if t < c["first"] or t >= x - c["recent"]]
        rest = np.setdiff1d(np.arange(x), must)
        rest = rest[np.argsort(-mass[a, rest], kind="stable")][: max(0, c["budget"] - len(must))]
        idx = np.sort(np.concatenate([np.asarray(must, np.int64), rest]))
        row, was = table[a], table[a].copy()
        shift = np.nonzero(idx != np.arange(len(idx)))[0]
        nb_new, nb_old = -(-len(idx) // block), -(-x // block)
        for b in range(shift[0] // block if len(shift) else nb_new, nb_new):
            if start[was[b]] > 1:
                row[b] = free.pop()
                refs[row[b]] = 1
                gone.append(was[b])
        gone += was[nb_new:nb_old].tolist()
        row[nb_new:nb_old] = -1
        i = np.arange(len(idx))
        moves.append((row[i // block], i % block, was[idx // block], idx % block))
        mass[a, :len(idx)] = mass[a, idx]
        mass[a, len(idx):x] = 0.0
        lists.append(idx)
    np.subtract.at(refs, np.asarray(gone, np.int64), 1)
    n_free = len(free) + int(((start > 0) & (refs == 0)).sum())
    to, at, src, sat = (torch.as_tensor(np.concatenate(x), device="cuda").long() for x in zip(*moves))
    out = {"idx": s["idx"].clone(), "idx_off": torch.as_tensor(np.concatenate([[0], np.cumsum([len(x) for x in lists])])),
           "table": table, "seq_len": np.array([len(x) for x in lists], np.int32), "refcount": refs,
           "n_free": np.array([n_free], np.int32), "mass": mass}
    got = np.concatenate(lists)
    out["idx"][: len(got)] = torch.as_tensor(got, device="cuda").int()
    for name in ("k", "v", "ksc", "vsc"):
        out[name] = [x.clone() if x is not None else None for x in s[name]]
        for x, y in zip(out[name], s[name]):
            if x is not None:
                x[to, :, at] = y[src, :, sat]
        if c["pool"] == "bf16":
            out[name] = [x.double() if x is not None else None for x in out[name]]
    return out
