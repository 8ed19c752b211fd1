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


