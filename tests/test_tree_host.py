"""Refusals of the tree attention, of the rotary append by axes and of the compaction, and the block
manager's truncation, without a GPU."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_207_gb300 import build, _native
    build.build()
    return _native


def _tree(L, **kw):
    a = dict(out=16, q=16, k=16, v=16, tables=16, mb=4, start=16, cu=16, mask=16, words=1, S=1, T=4, chunk=4, Hq=4, Hkv=2,
             D=64, nb=8, scale=0.125, dtype=1, ws=16, wsb=1 << 30)
    a.update(kw)
    return L.pa_tree_attention(*a.values(), None, None)


def test_tree_attention_refusals(native):
    L = native.lib()
    assert _tree(L, S=0) == OK and _tree(L, T=0) == OK and _tree(L, chunk=0) == OK
    for name in ("out", "q", "k", "v", "tables", "start", "cu", "mask", "ws"):
        assert _tree(L, **{name: None}) == INVALID, name
    for name in ("out", "q", "k", "v", "ws"):
        assert _tree(L, **{name: 24}) == INVALID, name
    assert _tree(L, dtype=4) == INVALID and _tree(L, dtype=-1) == INVALID
    assert _tree(L, D=96) == UNSUPPORTED and _tree(L, Hq=18) == UNSUPPORTED and _tree(L, Hq=5) == INVALID
    assert _tree(L, scale=float("nan")) == INVALID and _tree(L, scale=float("inf")) == INVALID
    assert _tree(L, mb=2**27) == INVALID and _tree(L, mb=0) == INVALID and _tree(L, nb=0) == INVALID
    for name in ("S", "T", "chunk", "words"):
        assert _tree(L, **{name: -1}) == INVALID, name
    assert _tree(L, Hkv=0) == INVALID and _tree(L, Hq=0) == INVALID
    # a mask narrower than the trees, and a workspace smaller than they need
    assert _tree(L, T=40, chunk=33) == INVALID and _tree(L, T=40, chunk=2**31 - 1) == INVALID
    need = L.pa_tree_workspace_size(4, 2, 64, 4)
    assert need > 0 and _tree(L, wsb=need - 1) == INVALID


def test_tree_workspace_size(native):
    size = native.tree_workspace_size
    assert size(4, 2, 64, 0) == 0 and size(4, 2, 64, -3) == 0 and size(4, 3, 64, 5) == 0 and size(18, 2, 64, 5) == 0
    assert 0 < size(4, 2, 64, 1) <= size(4, 2, 64, 8) <= size(4, 2, 64, 64) <= size(4, 2, 64, 10**6)
    assert size(4, 2, 64, 10**6) == size(4, 2, 64, 2**40)          # a group of rows at a time, whatever the trees
    assert size(32, 8, 128, 64) % 16 == 0


def _compact(L, **kw):
    a = dict(k=16, v=16, tables=16, mb=4, src=16, start=16, cu=16, dst=32, dmb=4, S=1, T=4, nb=8, Hkv=2, D=64, dtype=1)
    a.update(kw)
    return L.pa_compact_kv(*a.values(), None, None)


def test_compact_refusals(native):
    L = native.lib()
    assert _compact(L, S=0) == OK and _compact(L, T=0) == OK
    for name in ("k", "v", "tables", "src", "start", "cu"):
        assert _compact(L, **{name: None}) == INVALID, name
    for name in ("k", "v"):
        assert _compact(L, **{name: 24}) == INVALID, name
    assert _compact(L, dtype=4) == INVALID and _compact(L, D=96) == UNSUPPORTED
    assert _compact(L, mb=0) == INVALID and _compact(L, mb=2**27) == INVALID
    assert _compact(L, dmb=0) == INVALID and _compact(L, dmb=2**27) == INVALID
    assert _compact(L, dst=16, dmb=5) == INVALID                # the same table with another width
    assert _compact(L, S=65536) == UNSUPPORTED and _compact(L, Hkv=65536) == UNSUPPORTED
    assert _compact(L, S=-1) == INVALID and _compact(L, T=-1) == INVALID and _compact(L, nb=0) == INVALID


def _axes(L, **kw):
    a = dict(kp=16, vp=16, qo=32, q=16, kn=16, vn=16, qos=256, qs=256, ks=128, vs=128, freq=16, R=64, il=0, pos=16, axes=3,
             plane=16, tables=16, mb=4, start=16, cu=16, S=1, T=2, nb=8, Hq=4, Hkv=2, D=64, dtype=1)
    a.update(kw)
    return L.pa_rope_append_kv_axes(*a.values(), None, None)


def test_rope_axes_refusals(native):
    L = native.lib()
    assert _axes(L, S=0, T=0) == OK
    assert _axes(L, axes=0) == INVALID and _axes(L, axes=-1) == INVALID
    assert _axes(L, pos=None) == INVALID and _axes(L, plane=None) == INVALID
    assert _axes(L, axes=1, plane=None, kn=None) == INVALID
    for name in ("kp", "vp", "kn", "vn", "freq", "tables", "start", "cu"):
        assert _axes(L, **{name: None}) == INVALID, name
    assert _axes(L, q=None) == INVALID and _axes(L, R=24) == UNSUPPORTED and _axes(L, R=80) == INVALID
    assert _axes(L, ks=127) == INVALID and _axes(L, dtype=7) == INVALID and _axes(L, D=96) == UNSUPPORTED


def test_bindings_check_the_tensors(native):
    bf16, i32 = torch.bfloat16, torch.int32
    pool = torch.zeros(native.pool_shape(4, 2, 64, bf16), dtype=bf16)
    q, new = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tables, lens, cu = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32), torch.arange(4, dtype=i32)
    mask, ws = torch.ones(3, 1, dtype=i32), torch.zeros(1 << 10, dtype=torch.uint8)
    freq, pos, plane = torch.ones(32, dtype=torch.float64), torch.zeros(2, 3, dtype=i32), torch.zeros(32, dtype=i32)
    with pytest.raises(ValueError):                              # on the host
        native.tree_attention(q.clone(), q, pool, pool, tables, lens, cu, mask, 0.1, 1, ws)
    with pytest.raises(ValueError):
        native.tree_attention(q.clone(), q, pool, pool, tables, lens, cu, mask[0], 0.1, 1, ws)
    with pytest.raises(ValueError):
        native.tree_attention(q.clone(), q[0], pool, pool, tables, lens, cu, mask, 0.1, 1, ws)
    with pytest.raises(TypeError):
        native.tree_attention(q.clone(), q, pool.half(), pool.half(), tables, lens, cu, mask, 0.1, 1, ws)
    with pytest.raises(ValueError):
        native.compact_kv(pool, pool, tables, lens, lens, cu)
    with pytest.raises(ValueError):
        native.compact_kv(pool, pool, tables[0], lens, lens, cu)
    with pytest.raises(ValueError):
        native.compact_kv_fp8(pool, pool, tables, lens, lens, cu)
    with pytest.raises(ValueError):
        native.rope_append_kv_axes(pool, pool, q.clone(), q, new, new, freq, plane, pos, tables, lens, cu)
    with pytest.raises(ValueError):
        native.rope_append_kv_axes(pool, pool, None, q, new, new, freq, plane, pos, tables, lens, cu)


def test_truncate(native):
    bm = native.BlockManager(8)
    a = bm.add_seq()
    bm.prepare_append(a, 0, 50)                                   # four blocks
    b = bm.fork(a)
    row = bm.block_table(a, 4)
    bm.truncate(a, 33)                                            # three of them
    assert bm.seq_len(a) == 33 and bm.block_table(a, 4) == row[:3] + [-1]
    assert [bm.refcount(x) for x in row] == [2, 2, 2, 1]          # the fork keeps the last
    bm.truncate(a, 33)
    bm.truncate(a, 32)
    assert bm.block_table(a, 4) == row[:2] + [-1, -1] and bm.seq_len(b) == 50
    assert bm.stats()["logical_tokens"] == 82
    bm.truncate(b, 0)
    assert [bm.refcount(x) for x in row] == [1, 1, 0, 0] and bm.stats()["free_blocks"] == 6
    bm.truncate(a, 0)
    assert bm.stats()["free_blocks"] == 8 and bm.stats()["logical_tokens"] == 0
    bm.prepare_append(a, 0, 1)
    assert bm.block_table(a, 1) == [0]                            # lowest first, as ever
    for bad in ((a, 2), (a, -1), (99, 0)):
        with pytest.raises(native.PagedKVError):
            bm.truncate(*bad)
    assert bm.seq_len(a) == 1
