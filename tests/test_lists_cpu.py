"""Lists of kept tokens: the binding passes their length on, and no pool is refused (no GPU is needed)."""
import types

import pytest

torch = pytest.importorskip("torch")

from shared_paged_kv_gb300 import kvs as K
from test_binding_devices import On


class Pool:
    handle, desc = 1, types.SimpleNamespace(num_kv_heads=2, head_dim=64, block_tokens=16, capacity_blocks=8)


@pytest.mark.parametrize("n", [0, 1, 77])
def test_the_lists_length_is_passed_on(monkeypatch, n):
    seen = {}
    lib = types.SimpleNamespace(kvs_keep_heavy_bounded=lambda *a: seen.update(keep=a) or 0,
                                kvs_compact_bounded=lambda *a: seen.update(compact=a) or 0)
    monkeypatch.setattr(K, "_cur_dev", lambda: 0)
    monkeypatch.setattr(K, "load", lambda: lib)
    monkeypatch.setattr(K, "_stream", lambda s: None)
    i32, i64, f32 = (lambda *s: On(0, torch.int32, *s)), (lambda *s: On(0, torch.int64, *s)), (lambda *s: On(0, torch.float32, *s))
    K.kvs_keep_heavy(Pool, f32(2, 64), i32(2), 2, 4, i32(2), 1, 1, i32(n), i64(3))
    assert seen["keep"][9] == n
    K.kvs_compact(Pool, i32(2, 4), 4, i32(2), 2, i32(n), i64(3), i32(8), i32(8), i32(1), On(0, torch.uint8, 1 << 12))
    assert seen["compact"][6] == n


def test_no_pool():
    import __graft_entry__ as g
    g.build()
    lib = K.load()
    assert lib.kvs_keep_heavy_bounded(None, None, None, 1, 1, None, 0, 0, None, 0, None, None) == K.KVS_ERR_INVALID_ARG
    assert lib.kvs_compact_bounded(None, None, 1, None, 1, None, 0, None, None, None, None, None, None, 0, None) == K.KVS_ERR_INVALID_ARG
