"""The operators that make room, one after the other as a model's loop calls them: prompts go into the pool, their last
rows (or a few decode steps) gather the tokens' weights over the layers, every sequence keeps its heaviest tokens, and
decoding goes on over what is left, with the tokens' true positions.  Every step is compared with the fp64 oracle on what
the pool holds before it."""
import numpy as np
import pytest
import torch

from oracle import compact as OC
from oracle import mass as OM
from oracle import mx4 as O4
from shared_paged_kv_gb300 import kvs as K

from harness import DEV, i32, workspace

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


class Model:
    """Layers, pool and tables of a few sequences; the last one is a fork of the one before it."""

    def __init__(self, kind, lens, hq, hkv, d, layers, seed=0):
        self.kind, self.hq, self.hkv, self.d, self.layers, self.n = kind, hq, hkv, d, layers, len(lens)
        self.block = {"bf16": 16, "mx4": 64}[kind]
        self.g, r = torch.Generator(device=DEV).manual_seed(seed), np.random.default_rng(seed)
        nb = [-(-x // self.block) + 1 for x in lens]      # one to grow into
        self.mb, self.cap = max(nb), sum(nb[:-1]) + 40
        ids, at = r.permutation(self.cap), 0
        table, refs = np.full((self.n, self.mb), -1), np.zeros(self.cap, np.int64)
        for a in range(self.n - 1):
            table[a, :nb[a]] = ids[at:at + nb[a]]
            at += nb[a]
        table[-1, :nb[-1] - 1] = table[-2, :nb[-1] - 1]
        refs[table[:-1][table[:-1] >= 0]] = 1
        refs[table[-1, :nb[-1] - 1]] += 1
        free = np.sort(ids[at:])[::-1]
        self.table, self.lens, self.refs, self.n_free = i32(table), i32(lens), i32(refs), i32([len(free)])
        self.free = i32(np.concatenate([free, np.zeros(self.cap - len(free))]))
        full = lambda w, dt: [torch.randint(0, 255, (self.cap, hkv, self.block, w), generator=self.g, device=DEV, dtype=torch.uint8).view(dt)  # noqa: E731
                              for _ in range(layers)]
        if kind == "bf16":
            self.k, self.v = ([torch.zeros(self.cap, hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(layers)] for _ in range(2))
            self.slabs = [x for pair in zip(self.k, self.v) for x in pair]
            self.pool = K.kvs_pool_create(layers, hkv, d, 16, K.KVS_DTYPE_BF16, self.cap, self.n, self.k, self.v)
        else:
            self.k, self.v, self.ks, self.vs = full(64, torch.uint8), full(64, torch.uint8), full(4, torch.uint8), full(4, torch.uint8)
            self.slabs = [x for four in zip(self.k, self.v, self.ks, self.vs) for x in four]
            self.pool = K.kvs_pool_create(layers, hkv, d, 64, K.KVS_DTYPE_MX4, self.cap, self.n, self.k, self.v, self.ks, self.vs)
        self.mass = torch.zeros(self.n, self.mb * self.block, device=DEV)
        self.rope = K.RopeAxes(1e4, (d // 2,))
        self.place = np.array(lens)                       # true positions to come

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV).to(torch.bfloat16)

    def values(self, layer):
        if self.kind == "bf16":
            return f64(self.k[layer]), f64(self.v[layer])
        return (O4.dequantize(self.k[layer].cpu().numpy(), self.ks[layer].cpu().numpy()),
                O4.dequantize(self.v[layer].cpu().numpy(), self.vs[layer].cpu().numpy()))

    def append(self, layer, new, pos):
        """new[a] more rows of every sequence (counted in self.lens already); the rotated queries."""
        off, T = i32(np.concatenate([[0], np.cumsum(new)])), int(sum(new))
        k, v, q = self.randn(T, self.hkv, self.d), self.randn(T, self.hkv, self.d), self.randn(T, self.hq, self.d)
        q_rot = torch.empty_like(q)
        K.kvs_append(self.pool, layer, k, v, T, off, self.table, self.mb, self.lens, self.n, pos=pos, rope=self.rope, q=q,
                     n_q_heads=self.hq, q_out=q_rot)
        return off, T, q_rot

    def add(self, layer, q, off, T, causal):
        """The weights of T rows (the last of every sequence), added in place and compared."""
        before, n, scale = f64(self.mass), self.n, self.d ** -0.5
        K_, V = self.values(layer)
        lens = self.lens.tolist()
        out = None
        if causal:
            ws = workspace(K.kvs_extend_mass_workspace_size(self.pool, T, n, self.mb, self.hq))
            K.kvs_extend_mass(self.pool, layer, q, T, off, self.hq, self.table, self.mb, self.lens, n, True, scale, self.mass, 1.0,
                              self.mass, ws)
        else:
            out = torch.empty(n, self.hq, self.d, device=DEV)
            ws = workspace(K.kvs_workspace_size(self.pool, K.KVS_OP_DECODE_MASS, n, self.mb, self.hq))
            if self.kind == "bf16":
                K.kvs_decode_attn_mass(self.pool, layer, q, self.hq, self.table, self.mb, self.lens, n, scale, out, self.mass, 1.0,
                                       self.mass, ws)
            else:
                K.kvs_decode_attn_mx4(self.pool, layer, q, self.hq, self.table, self.mb, self.lens, n, scale, out, ws,
                                      mass_in=self.mass, mass=self.mass)
        want, _, w, _ = OM.attend(f64(q), K_, V, self.table.cpu().numpy(), off.cpu().numpy(), lens, self.block, scale, causal)
        for a in range(n):
            np.testing.assert_allclose(f64(self.mass)[a, :lens[a]], before[a, :lens[a]] + w[a], rtol=1e-4, atol=1e-7)
        if out is not None:
            assert np.linalg.norm(f64(out) - want) <= 2e-5 * np.linalg.norm(want)

    def evict(self, budget, first, recent):
        mass, lens = self.mass.cpu().numpy(), self.lens.tolist()
        idx = torch.zeros(sum(lens), dtype=torch.int32, device=DEV)
        off = torch.zeros(self.n + 1, dtype=torch.int64, device=DEV)
        want_idx, want_off = OC.keep_heavy(mass, lens, budget, first, recent)
        want = OC.compact([s.cpu().view(torch.int16 if self.kind == "bf16" else torch.uint8).numpy() for s in self.slabs],
                          self.table.cpu().numpy(), lens, want_idx, want_off, mass, self.refs.cpu().numpy(),
                          self.free[: int(self.n_free)].tolist(), self.block)
        ws = workspace(K.kvs_workspace_size(self.pool, K.KVS_OP_COMPACT, self.n, self.mb))
        K.kvs_keep_heavy(self.pool, self.mass, self.lens, self.n, self.mb, i32(budget), first, recent, idx, off)
        K.kvs_compact(self.pool, self.table, self.mb, self.lens, self.n, idx, off, self.refs, self.free, self.n_free, ws, mass=self.mass)
        assert idx[: len(want_idx)].tolist() == want_idx.tolist()
        for got, exp in zip(self.slabs, want[0]):
            np.testing.assert_array_equal(got.cpu().view(torch.int16 if self.kind == "bf16" else torch.uint8).numpy(), exp)
        for got, exp in ((self.table, want[1]), (self.lens, want[2]), (self.mass, want[3]), (self.refs, want[4])):
            np.testing.assert_array_equal(got.cpu().numpy(), exp)
        assert self.free[: int(self.n_free)].tolist() == want[5] and want[6] == []

    def step(self):
        """One more token each, at its true position, in every layer."""
        self.lens += 1
        pos = i32(self.place)
        for layer in range(self.layers):
            off, T, q = self.append(layer, [1] * self.n, pos)
            self.add(layer, q, off, T, False)
        self.place += 1


@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 64), (4, 4, 128), (16, 1, 128)])
def test_prompts_window_eviction_and_decoding(hq, hkv, d):
    lens = [150, 301, 44, 44]
    m = Model("bf16", lens, hq, hkv, d, 2)
    prompt = [150, 301, 44, 0]                            # the fork has its parent's rows already
    for layer in range(2):
        off, T, q = m.append(layer, prompt, None)
        window = [16, 16, 16, 0]
        rows = torch.cat([torch.arange(int(o) - w, int(o)) for o, w in zip(off.tolist()[1:], window)]).to(DEV)
        m.add(layer, q[rows].contiguous(), i32(np.concatenate([[0], np.cumsum(window)])), sum(window), True)
    m.mass[3] = torch.rand(m.mb * 16, generator=m.g, device=DEV)   # the fork has a mind of its own
    m.evict([70, 135, 37, 20], 4, 8)
    for _ in range(3):
        m.step()
    m.evict([40, 60, 30, 100], 4, 8)
    m.step()
    assert K.kvs_pool_check(m.pool) == 0


def test_microscaled_prompts_decoding_and_eviction():
    lens = [150, 501, 200, 200]
    m = Model("mx4", lens, 8, 2, 128, 2)
    for layer in range(2):
        m.append(layer, [150, 501, 200, 0], None)
    # the fork's next token lies in a block that its parent has too: it gets its own copy first
    ws = workspace(K.kvs_workspace_size(m.pool, K.KVS_OP_BLOCKS, 4, m.mb))
    K.kvs_block_write(m.pool, m.table, m.mb, 4, i32([3]), i32([200 // 64]), 1, m.refs, m.free, m.n_free, ws)
    for _ in range(3):
        m.step()
    m.evict([100, 250, 70, 130], 2, 16)
    for _ in range(3):
        m.step()
    assert K.kvs_pool_check(m.pool) == 0
