"""Calls around drafted trees that are easily made by mistake: what they refuse or flag, and what they leave as it was."""
import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _tree_common import ancestors, attention, moved, packed, random_tree, rng_of, visible
from _window_common import Cache, nan_like, unpacked, within

pytestmark = pytest.mark.gpu

CACHES = ["bf16", "f32", "fp8", "fp4"]


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def of_cache(name, cache):
    return getattr(pk, name + {"fp8": "_fp8", "fp4": "_fp4"}.get(cache, ""))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("quick", [True, False])
def test_compaction_into_a_table_without_columns(cache, quick, monkeypatch):
    # refused, and not taken for one in place
    pk.lib()
    if not quick:
        monkeypatch.setattr(pk._native, "_quick", None)
    c = Cache(cache, [40, 20], (2, 2, 64), seed=70)
    before = c.kp.clone(), c.vp.clone()
    none = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    with pytest.raises((ValueError, pk.PagedKVError)):
        of_cache("compact_kv", cache)(c.kp, c.vp, c.tables.cuda(), i32([30, 31, 10]), i32([0, 2]), i32([0, 2, 3]), dst_tables=none)
    torch.cuda.synchronize()
    for was, now in zip(before, (c.kp, c.vp)):
        assert torch.equal(was.view(torch.uint8), now.view(torch.uint8))
    # without rows there is nothing to refuse
    of_cache("compact_kv", cache)(c.kp, c.vp, c.tables.cuda(), i32([]), i32([0, 2]), i32([0, 0, 0]), dst_tables=none)


@pytest.mark.parametrize("cache", CACHES)
def test_a_bound_of_no_nodes(cache):
    # like any other that is too small: the nodes are flagged, and not computed
    c = Cache(cache, [20, 12], (4, 2, 64), seed=71)
    q = c.queries(5).cuda()
    mask, ws = torch.ones(5, 1, dtype=torch.int32, device="cuda"), pk.tree_workspace(4, 2, 64, 0)

    def call(cu):
        out, err = nan_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        of_cache("tree_attention", cache)(out, q, c.kp, c.vp, c.tables.cuda(), i32([10, 10]), i32(cu), mask, 0.1, 0, ws, err_flag=err)
        assert bool(out.isnan().all())
        return int(err)

    assert call([0, 3, 5]) == pk.DEV_ERR_HINT
    assert call([0, 0, 2]) == pk.DEV_ERR_HINT
    assert call([0, 0, 0]) == 0
    assert call([0, 7, 7]) == pk.DEV_ERR_BAD_CU
    out = nan_like(q)                                                # without a flag
    of_cache("tree_attention", cache)(out, q, c.kp, c.vp, c.tables.cuda(), i32([10, 10]), i32([0, 3, 5]), mask, 0.1, 0, ws)
    assert bool(out.isnan().all())


@pytest.mark.parametrize("cache", CACHES)
def test_compaction_of_refused_sequences_moves_the_others(cache):
    lens = [40, 40, 40]
    heads = (2, 2, 64)
    for cu, good in (([0, 2, 1, 3], {0: [30, 31], 2: [31, 32]}), ([-1, 1, 2, 3], {1: [31], 2: [32]}), ([0, 1, 2, 9], {0: [30], 1: [31]}),
                     ([0, 2, 2, 3], {0: [30, 31], 2: [32]})):
        c = Cache(cache, lens, heads, seed=72)
        before = [unpacked(cache, t, 64, keys) for t, keys in ((c.kp, True), (c.vp, False))]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        of_cache("compact_kv", cache)(c.kp, c.vp, c.tables.cuda(), i32([30, 31, 32]), i32([0, 0, 0]), i32(cu), err_flag=err)
        assert int(err) == (0 if cu == [0, 2, 2, 3] else pk.DEV_ERR_BAD_CU)
        src = [good.get(s, []) for s in range(3)]
        for was, (t, keys) in zip(before, ((c.kp, True), (c.vp, False))):
            assert torch.equal(moved(was, c.tables, c.tables, src, [0, 0, 0]), unpacked(cache, t, 64, keys)), (cu, keys)


@pytest.mark.parametrize("cache", CACHES)
def test_trees_beside_refused_ones(cache):
    # a falling offset: the sequence that it begins or ends is refused, the others are computed
    c = Cache(cache, [40, 40, 40], (4, 2, 64), seed=73)
    rng = rng_of("beside", cache)
    sees = [ancestors(random_tree(8, rng)) for _ in range(3)]
    q = c.queries(24)
    ws, err = pk.tree_workspace(4, 2, 64, 8), torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu, flags, good in (([0, 8, 5, 13], pk.DEV_ERR_BAD_CU, [0]), ([16, 8, 16, 24], pk.DEV_ERR_BAD_CU, [1, 2]),
                            ([0, 8, 16, 25], pk.DEV_ERR_BAD_CU, [0, 1])):
        out = nan_like(q.cuda())
        err.zero_()
        of_cache("tree_attention", cache)(out, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32([32] * 3), i32(cu), packed(sees).cuda(), 0.1, 8,
                                          ws, err_flag=err)
        assert int(err) == flags
        for s in range(3):
            rows = slice(8 * s, 8 * s + 8)
            if s in good:
                at = slice(cu[s], cu[s] + 8) if cu[s + 1] - cu[s] == 8 else None
                want, tol = attention(q[at], c.k[s], c.v[s], visible(32, sees[cu[s] // 8]), 0.1, cache, q.dtype)
                # (rows that a later chunk, of other rows, does not write too)
                mine = slice(at.start, min([at.stop] + [cu[x] for x in range(s + 1, 3) if at.start < cu[x] < at.stop and cu[x + 1] > cu[x]]))
                n = mine.stop - mine.start
                within(out[mine], want[:n], tol[:n], f"sequence {s} of {cu}")
        written = torch.zeros(24, dtype=torch.bool)
        for s in range(3):
            if 0 <= cu[s] <= cu[s + 1] <= 24:
                written[cu[s]:cu[s + 1]] = True
        assert bool(out[~written.cuda()].isnan().all())
