"""Tree attention, the rotary append by positions on axes and the compaction against plain 64-bit
implementations (tests/_tree_common.py, which derives the tolerances)."""
import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _tree_common import ancestors, attention, moved, packed, random_tree, rng_of, visible
from _window_common import BLOCK, Cache, half_step, nan_like, pool_for, rope_call, rotated, unpacked, within

pytestmark = pytest.mark.gpu

HEADS = [(4, 4, 64), (14, 2, 64), (8, 1, 128), (8, 2, 128), (9, 3, 128)]
CACHES = ["bf16", "f32", "fp8", "fp4"]


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def err_flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tree_call(cache):
    return {"fp8": pk.tree_attention_fp8, "fp4": pk.tree_attention_fp4}.get(cache, pk.tree_attention)


def compact_call(cache):
    return {"fp8": pk.compact_kv_fp8, "fp4": pk.compact_kv_fp4}.get(cache, pk.compact_kv)


def axes_call(cache):
    return {"fp8": pk.rope_append_kv_axes_fp8, "fp4": pk.rope_append_kv_axes_fp4}.get(cache, pk.rope_append_kv_axes)


def cumulated(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


# ---------------------------------------------------------------------------- tree attention
def run_tree(c, ctx, sees, q, scale, err=None, out=None, words=None, max_chunk=None, workspace=None, **kw):
    out = nan_like(q.cuda()) if out is None else out
    counts = [x.shape[0] for x in sees]
    chunk = max(counts) if max_chunk is None else max_chunk
    ws = pk.tree_workspace(c.hq, c.hkv, c.d, chunk) if workspace is None else workspace
    tree_call(c.cache)(out, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(ctx), i32(cumulated(counts)),
                       packed(sees, words).cuda(), scale, chunk, ws, err_flag=err, **kw)
    return out


def check_tree(c, ctx, sees, q, scale, out):
    cu = cumulated([x.shape[0] for x in sees])
    for s, (a, see) in enumerate(zip(ctx, sees)):
        n = see.shape[0]
        if n == 0:
            continue
        rows = slice(cu[s], cu[s + 1])
        want, tol = attention(q[rows], c.k[s][:a + n], c.v[s][:a + n], visible(a, see), scale, c.cache, q.dtype)
        within(out[rows], want, tol, f"sequence {s}: {n} nodes after {a}")


def trees(counts, *key):
    rng = rng_of(*key)
    return [ancestors(random_tree(n, rng)) for n in counts]


def poison_ends(c, ctx, sees):
    for s, (a, see) in enumerate(zip(ctx, sees)):
        c.poison(s, [True] * (a + see.shape[0]))


CTX = [0, 1, 15, 16, 17, 100, 257, 130, 0, 64]
NODES = [1, 5, 16, 17, 33, 3, 2, 40, 7, 0]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", HEADS)
def test_tree_attention(cache, heads):
    sees = trees(NODES, cache, heads)
    sees[8][3:5] = False                       # rows that see nothing at all
    sees[3][2] = False                         # and one that sees its context alone
    c = Cache(cache, [a + n for a, n in zip(CTX, NODES)], heads, seed=1)
    poison_ends(c, CTX, sees)
    q = c.queries(sum(NODES))
    err = err_flag()
    out = run_tree(c, CTX, sees, q, heads[2] ** -0.5, err)
    assert int(err) == 0
    check_tree(c, CTX, sees, q, heads[2] ** -0.5, out)
    first = sum(NODES[:8])
    assert bool((out[first + 3:first + 5] == 0).all())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(8, 1, 128), (4, 4, 64), (7, 1, 64)])
def test_wide_trees(cache, heads):
    ctx, nodes = [40, 0, 200], [100, 33, 64]
    sees = trees(nodes, cache, heads)
    c = Cache(cache, [a + n for a, n in zip(ctx, nodes)], heads, seed=2)
    q = c.queries(sum(nodes))
    out = run_tree(c, ctx, sees, q, 0.1)
    check_tree(c, ctx, sees, q, 0.1, out)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("nodes", [1, 9, 40])
def test_long_contexts_over_many_ctas(cache, nodes):
    ctx, counts = [9000, 3, 4111], [nodes, 2, nodes]
    sees = trees(counts, cache, nodes)
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (8, 2, 128), seed=3)
    poison_ends(c, ctx, sees)
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, 0.09)
    check_tree(c, ctx, sees, q, 0.09, out)


@pytest.mark.parametrize("cache", CACHES)
def test_many_short_sequences(cache):
    # more items than CTAs, several of them a CTA's, empty ones between
    rng = rng_of("many", cache)
    ctx = [rng.randint(0, 300) for _ in range(230)]
    counts = [rng.choice([0, 1, 2, 5, 11]) for _ in ctx]
    sees = trees(counts, "many", cache)
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (4, 2, 64), seed=4)
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, 0.125)
    check_tree(c, ctx, sees, q, 0.125, out)


@pytest.mark.parametrize("cache", CACHES)
def test_any_mask_is_a_mask(cache):
    # later nodes, all nodes, random ones; words wider than the trees with bits behind the last node
    rng = rng_of("masks")
    ctx, counts = [20, 300, 0], [50, 33, 20]
    sees = [torch.tensor([[rng.random() < 0.5 for _ in range(n)] for _ in range(n)]) for n in counts]
    sees[1][:] = True
    sees[2][:, :10] = False
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (4, 1, 128), seed=5)
    q = c.queries(sum(counts))
    mask = packed(sees, 4)
    row = 0
    for n in counts:                           # what is behind a sequence's last node does not matter
        for j in range(n, 128):
            mask[row:row + n, j // 32] |= 1 << (j % 32) if j % 32 < 31 else -2**31
        row += n
    out = nan_like(q.cuda())
    tree_call(cache)(out, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(ctx), i32(cumulated(counts)), mask.cuda(), 0.1, 50,
                     pk.tree_workspace(4, 1, 128, 50))
    check_tree(c, ctx, sees, q, 0.1, out)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_hidden_nodes_may_hold_anything(cache, what):
    # a node whose key and value are no finite numbers reaches the rows that see it and no others
    ctx, counts = [70, 130], [24, 40]
    sees = trees(counts, "hidden")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (8, 2, 128), seed=6)
    bad = [(0, 5), (0, 11), (1, 0), (1, 39)]
    for s, j in bad:
        p = ctx[s] + j
        blk, t = int(c.tables[s, p // BLOCK]), p % BLOCK
        if cache in ("bf16", "f32"):
            c.kp[blk, :, :, t, :] = what
            c.vp[blk, :, :, t, :] = what
        elif cache == "fp8" and what == what:   # scales of infinity: codes of zero give NaN, others an infinity
            for pool in (c.kp, c.vp):
                pool[blk, :, 16 * 128:].view(torch.float32)[:, t] = what
        else:
            c._poison_slot(c.kp[blk], t, True)
            c._poison_slot(c.vp[blk], t, False)
    c.refresh()
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, 0.1)
    cu = cumulated(counts)
    for s in range(2):
        hit = torch.zeros(counts[s], dtype=torch.bool)
        for x, j in bad:
            if x == s:
                hit |= sees[s][:, j]
        clean = torch.nonzero(~hit).flatten()
        assert 0 < len(clean) < counts[s]
        k, v = (x[s].clone() for x in (c.k, c.v))
        for x, j in bad:
            if x == s:
                k[ctx[s] + j] = v[ctx[s] + j] = 0.0              # (hidden from every clean row)
        want, tol = attention(q[cu[s] + clean], k, v, visible(ctx[s], sees[s][clean]), 0.1, cache, q.dtype)
        within(out[cu[s] + clean.cuda()], want, tol, f"rows that do not see them, sequence {s}")
        if cache != "fp4":
            assert not bool(torch.isfinite(out[cu[s] + torch.nonzero(hit).flatten().cuda()]).all(-1).any())


@pytest.mark.parametrize("cache", ["bf16", "f32", "fp8"])
def test_one_odd_value_of_a_node(cache):
    # a single element: the other dims of the rows that see it keep their values
    ctx, counts = [33], [20]
    sees = trees(counts, "odd")
    c = Cache(cache, [53], (4, 1, 128), seed=7)
    j, dim = 6, 77
    blk, t = int(c.tables[0, (33 + j) // BLOCK]), (33 + j) % BLOCK
    if cache == "fp8":
        c.vp[blk, 0, dim * 16 + t] = 0x7f
    else:
        X = c.vp.shape[-1]
        c.vp[blk, 0, dim // X, t, dim % X] = float("inf")
    q = c.queries(20)
    out = run_tree(c, ctx, sees, q, 0.1)
    v = c.v[0].clone()
    want, tol = attention(q, c.k[0], v, visible(33, sees[0]), 0.1, cache, q.dtype)
    others = [d for d in range(128) if d != dim]
    within(out[..., others], want[..., others], tol[..., others])
    hit = sees[0][:, j].cuda()
    assert not bool(torch.isfinite(out[hit][..., dim]).any())
    within(out[~hit][..., dim], want[~hit.cpu()][..., dim], tol[~hit.cpu()][..., dim])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("scale", [0.0, -0.2, 30.0])
def test_scales(cache, scale):
    ctx, counts = [150, 7], [20, 9]
    sees = trees(counts, "scales")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (4, 2, 64), seed=8)
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, scale)
    check_tree(c, ctx, sees, q, scale, out)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_keys_of_minus_infinity(cache):
    # scores of -inf weigh nothing; a row whose scores are all -inf gives zeros
    ctx, counts = [40], [6]
    c = Cache(cache, [46], (2, 1, 64), seed=9)
    blk, t = int(c.tables[0, 1]), 3
    c.kp[blk, :, :, t, :] = -float("inf")
    c.refresh()
    q = c.queries(6).abs() + 0.5               # (so that the score is -inf, not NaN)
    q = q.to(c.wide)
    sees = [torch.eye(6, dtype=torch.bool)]
    out = run_tree(c, ctx, sees, q, 0.1)
    see = visible(40, sees[0])
    see[:, 19] = False
    k = c.k[0].clone()
    k[19] = 0.0
    want, tol = attention(q, k, c.v[0], see, 0.1, cache, q.dtype)
    within(out, want, tol)
    c.kp.fill_(-float("inf"))
    assert bool((run_tree(c, ctx, sees, q, 0.1) == 0).all())


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_scales_far_apart(cache):
    # values and keys whose scales grow by 2^40 along the context, and shrink
    ctx, counts = [700], [12]
    heads = (4, 2, 128)
    c = Cache(cache, [712], heads, seed=10)
    g = torch.Generator().manual_seed(11)
    for up in (True, False):
        x = torch.linspace(-20, 20, 712) * (1 if up else -1)
        rows = [(torch.randn(712, 2, 128, generator=g) * torch.exp2(x)[:, None, None]).to(torch.bfloat16) for _ in (0, 1)]
        append = pk.append_kv_fp8 if cache == "fp8" else pk.append_kv_fp4
        append(c.kp, c.vp, (rows[0].float() * 2.0 ** -20).to(torch.bfloat16).cuda(), rows[1].cuda(), c.tables.cuda(), i32([0]), i32([0, 712]))
        c.refresh()
        sees = trees(counts, "far", up)
        q = c.queries(12)
        out = run_tree(c, ctx, sees, q, 0.1)
        check_tree(c, ctx, sees, q, 0.1, out)


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_queries_of_any_size(cache):
    c = Cache(cache, [90], (4, 2, 64), seed=12)
    sees = trees([10], "size")
    for e in (-100, -20, 60, 110):
        q = (c.queries(10).float() * 2.0 ** e).to(torch.bfloat16)
        out = run_tree(c, [80], sees, q, 2.0 ** -e / 8)
        check_tree(c, [80], sees, q, 2.0 ** -e / 8, out)


@pytest.mark.parametrize("cache", CACHES)
def test_bad_chunks_and_padding(cache):
    # rows past the last sequence and of refused chunks stay as they are
    c = Cache(cache, [40, 40, 40], (4, 2, 64), seed=13)
    sees = trees([8, 8, 8], "bad")
    q = c.queries(30)
    mask = torch.cat([packed(sees), torch.full((6, 1), -1, dtype=torch.int32)]).cuda()
    ws = pk.tree_workspace(4, 2, 64, 8)

    def call(start, cu, chunk=8, tables=None):
        out, err = nan_like(q.cuda()), err_flag()
        tree_call(cache)(out, q.cuda(), c.kp, c.vp, (c.tables if tables is None else tables).cuda(), i32(start), i32(cu), mask, 0.1,
                         chunk, ws, err_flag=err)
        return out, int(err)

    def fine(out, *seqs):
        for s in seqs:
            want, tol = attention(q[8 * s:8 * s + 8], c.k[s], c.v[s], visible(32, sees[s]), 0.1, cache, q.dtype)
            within(out[8 * s:8 * s + 8], want, tol, f"sequence {s}")

    out, err = call([32] * 3, [0, 8, 16, 24])
    assert err == 0 and bool(out[24:].isnan().all())
    fine(out, 0, 1, 2)
    for start in (-1, 41, 2**31 - 1, -2**31):
        out, err = call([32, start, 32], [0, 8, 16, 24])
        assert err == pk.DEV_ERR_BAD_POS and bool(out[8:16].isnan().all())
        fine(out, 0, 2)
    out, err = call([32] * 3, [0, 8, 16, 31])
    assert err == pk.DEV_ERR_BAD_CU and bool(out[16:].isnan().all())
    fine(out, 0, 1)
    out, err = call([32] * 3, [0, 8, 5, 24])
    assert err & pk.DEV_ERR_BAD_CU
    out, err = call([32] * 3, [-3, 8, 16, 24])
    assert err == pk.DEV_ERR_BAD_CU and bool(out[:8].isnan().all())
    fine(out, 1, 2)
    # nodes past the bound: neither computed nor seen
    out, err = call([32] * 3, [0, 8, 16, 24], chunk=5)
    assert err == pk.DEV_ERR_HINT
    for s in range(3):
        assert bool(out[8 * s + 5:8 * s + 8].isnan().all())
        want, tol = attention(q[8 * s:8 * s + 5], c.k[s][:37], c.v[s][:37], visible(32, sees[s][:5, :5]), 0.1, cache, q.dtype)
        within(out[8 * s:8 * s + 5], want, tol)
    for entry in (-1, c.blocks, 2**31 - 1):
        tables = c.tables.clone()
        tables[1, 1] = entry
        out, err = call([32] * 3, [0, 8, 16, 24], tables=tables)
        assert err == pk.DEV_ERR_BAD_BLOCK
        fine(out, 0, 2)


@pytest.mark.parametrize("cache", CACHES)
def test_a_raised_timeout_flag_stops_the_call(cache):
    c = Cache(cache, [400], (4, 2, 64), seed=14)
    q = c.queries(8)
    err = torch.full((1,), pk.DEV_ERR_TIMEOUT, dtype=torch.int32, device="cuda")
    assert bool(run_tree(c, [392], trees([8], 1), q, 0.1, err).isnan().all())
    err.zero_()
    out = run_tree(c, [392], trees([8], 1), q, 0.1, err)
    check_tree(c, [392], trees([8], 1), q, 0.1, out)


@pytest.mark.parametrize("cache", CACHES)
def test_equal_calls_graphs_and_streams(cache):
    ctx, counts = [3000, 50, 800], [12, 30, 1]
    sees = trees(counts, "graphs")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (8, 2, 128), seed=15)
    q = c.queries(sum(counts)).cuda()
    first = run_tree(c, ctx, sees, q, 0.1)
    assert torch.equal(first, run_tree(c, ctx, sees, q, 0.1))
    # captured with a workspace that another graph uses too, replayed over new queries and lengths
    ws = pk.tree_workspace(8, 2, 128, 30)
    static_q, start, out, out2 = q.clone(), i32(ctx), nan_like(q), nan_like(q)
    tables, cu, mask = c.tables.cuda(), i32(cumulated(counts)), packed(sees).cuda()

    def call(o):
        tree_call(cache)(o, static_q, c.kp, c.vp, tables, start, cu, mask, 0.1, 30, ws)

    graphs = []
    for o in (out, out2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    for g in graphs:
        g.replay()
    assert torch.equal(out, first) and torch.equal(out2, first)
    static_q.copy_(c.queries(sum(counts)))
    start.copy_(i32([2100, 7, 0]))
    for g in graphs:
        g.replay()
    check_tree(c, [2100, 7, 0], sees, static_q.cpu(), 0.1, out)
    assert torch.equal(out, out2)
    # another stream, given or current, each with its own workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = run_tree(c, ctx, sees, q, 0.1)
    b = run_tree(c, ctx, sees, q, 0.1, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, first) and torch.equal(b, first)


def test_a_chain_is_a_causal_chunk():
    # a tree that is one path: the prefill of the same rows
    ctx, counts = [100, 513], [30, 64]
    sees = [torch.ones(n, n).tril().bool() for n in counts]
    c = Cache("bf16", [a + n for a, n in zip(ctx, counts)], (8, 2, 128), seed=16)
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, 0.1)
    check_tree(c, ctx, sees, q, 0.1, out)
    chunk = nan_like(q.cuda())
    pk.prefill_attention(chunk, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(ctx), i32(cumulated(counts)), 0.1, 64)
    check_tree(c, ctx, sees, q, 0.1, chunk)


# ---------------------------------------------------------------------------- rotary append by axes
def frequencies(rotary, base=10000.0):
    return (base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).cuda()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 0, 23], [700, 333, 64]])
def test_axes_that_hold_the_places_are_the_plain_append(cache, counts):
    heads, ctx = (8, 2, 128), [3, 40, 1000]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=20)
    n = sum(counts)
    x = torch.randn(n, 12, 128, generator=c.g).to(c.wide).cuda()
    q, k, v = torch.split(x, (8, 2, 2), dim=1)
    place = torch.tensor([a + i for a, m in zip(ctx, counts) for i in range(m)], dtype=torch.int32, device="cuda")
    plane = i32([f % 3 for f in range(32)])
    for interleaved in (False, True):
        kp, vp, kp2, vp2, kp3, vp3 = (t.clone() for t in (c.kp, c.vp) * 3)
        out, out2, out3 = (torch.empty(n, 8, 128, dtype=c.wide, device="cuda") for _ in range(3))
        rest = (c.tables.cuda(), i32(ctx), i32(cumulated(counts)), interleaved)
        rope_call(cache)(kp, vp, out, q, k, v, frequencies(64), *rest)
        err = err_flag()
        axes_call(cache)(kp2, vp2, out2, q, k, v, frequencies(64), plane, place.expand(3, n).contiguous(), *rest, err_flag=err)
        axes_call(cache)(kp3, vp3, out3, q, k, v, frequencies(64), None, place[None], *rest, err_flag=err)
        assert int(err) == 0
        for a, b in ((kp, kp2), (vp, vp2), (out, out2), (kp, kp3), (vp, vp3), (out, out3)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("rotary,interleaved", [(64, False), (64, True), (48, False), (32, True)])
@pytest.mark.parametrize("counts", [[4, 9], [800, 300]])
def test_axes_turn_their_planes(cache, rotary, interleaved, counts):
    heads, ctx = (4, 2, 64), [30, 5]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=21)
    n, half = sum(counts), rotary // 2
    q, k, v = (torch.randn(n, h, 64, generator=c.g).to(c.wide) for h in (4, 2, 2))
    rng = rng_of("axes", rotary)
    pos = torch.tensor([[rng.choice([0, -5, 7, 131071, 2**22 - 1, -2**22, rng.randint(0, 5000)]) for _ in range(n)] for _ in range(3)])
    plane = [rng.randrange(3) for _ in range(half)]
    freq = frequencies(rotary)
    out = nan_like(q.cuda())
    axes_call(cache)(c.kp, c.vp, out, q.cuda(), k.cuda(), v.cuda(), freq, i32(plane), pos.to(torch.int32).cuda(), c.tables.cuda(),
                     i32(ctx), i32(cumulated(counts)), interleaved)
    # a position of its own for each plane: one frequency at a time
    own = pos[torch.tensor(plane)].T.double() * freq.cpu()                 # [rows][half]: angles
    c.refresh()
    cu = cumulated(counts)
    for x, got in ((q, out.cpu()), (k, torch.cat([c.k[s][a:a + m] for s, (a, m) in enumerate(zip(ctx, counts))]))):
        want, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
        a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
        co, si = own.cos()[:, None], own.sin()[:, None]
        want[..., a] = x[..., a].double() * co - x[..., b].double() * si
        want[..., b] = x[..., b].double() * co + x[..., a].double() * si
        size[..., a] = size[..., b] = x[..., a].double().abs() + x[..., b].double().abs()
        within(got, want, half_step(c.wide) * want.abs() + 5e-7 * size * (1 + half_step(c.wide)) + 1e-30)
    assert torch.equal(torch.cat([c.v[s][a:a + m] for s, (a, m) in enumerate(zip(ctx, counts))]), v.double())
    assert cu[-1] == n


@pytest.mark.parametrize("counts", [[3, 2], [700, 10]])
def test_planes_without_an_axis_do_not_turn(counts):
    c = Cache("f32", counts, (2, 1, 64), seed=22)
    n = sum(counts)
    q, k, v = (torch.randn(n, h, 64, generator=c.g).cuda() for h in (2, 1, 1))
    pos = torch.randint(0, 1000, (2, n), generator=c.g, dtype=torch.int32).cuda()
    plane = [f % 2 for f in range(32)]
    good = torch.empty_like(q)
    rest = (c.tables.cuda(), i32([0, 0]), i32(cumulated(counts)))
    pk.rope_append_kv_axes(c.kp, c.vp, good, q, k, v, frequencies(64), i32(plane), pos, *rest)
    for bad in (-1, 2, 2**31 - 1, -2**31):
        out, err = torch.empty_like(q), err_flag()
        pk.rope_append_kv_axes(c.kp, c.vp, out, q, k, v, frequencies(64), i32(plane[:7] + [bad] + plane[8:]), pos, *rest, err_flag=err)
        assert int(err) == pk.DEV_ERR_BAD_POS
        assert torch.equal(out[..., [7, 39]], q[..., [7, 39]])
        rest_dims = [d for d in range(64) if d not in (7, 39)]
        assert torch.equal(out[..., rest_dims], good[..., rest_dims])


# ---------------------------------------------------------------------------- compaction
def pools_of(c):
    return [unpacked(c.cache, pool, c.d, keys) for pool, keys in ((c.kp, True), (c.vp, False))]


def check_moves(c, src, start, dst_tables=None, pad=0, expect=None):
    before = pools_of(c)
    counts = [len(x) for x in src]
    err = err_flag()
    compact_call(c.cache)(c.kp, c.vp, c.tables.cuda(), i32([p for x in src for p in x] + [-1] * pad), i32(start),
                          i32(cumulated(counts)), dst_tables=None if dst_tables is None else dst_tables.cuda(), err_flag=err)
    assert int(err) == 0
    to = c.tables if dst_tables is None else dst_tables
    for was, now in zip(before, pools_of(c)):
        assert torch.equal(moved(was, c.tables, to, src, start), now)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(1, 1, 64), (2, 2, 64), (3, 3, 128), (8, 8, 128)])
def test_compaction_in_place(cache, heads):
    lens = [0, 1, 40, 100, 3000, 17, 64]
    rng = rng_of("compact", cache, heads)
    c = Cache(cache, lens, heads, seed=30)
    start, src = [], []
    for n in lens:
        a = rng.randint(0, min(n, 20))
        start.append(a)
        keep = rng.choice([0.2, 0.5, 0.97])
        src.append([p for p in range(a, n) if rng.random() < keep])
    check_moves(c, src, start, pad=5)
    # every position again (nothing moves), one row, the last row to the front
    check_moves(c, [list(range(n)) for n in lens], [0] * len(lens))
    check_moves(c, [[n - 1] if n else [] for n in lens], [0] * len(lens))
    # the same row many times, and rows out of order, none from before its place
    src = [[], [0], [39] * 30, [99, 50, 98, 50, 51] + [99] * 40, [2999 - (i * 7) % 500 for i in range(2000)], [16, 3, 16], []]
    check_moves(c, src, [0, 0, 9, 33, 500, 1, 0])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(2, 2, 64), (3, 3, 128)])
def test_compaction_into_other_blocks(cache, heads):
    lens = [0, 5, 900, 33, 2500]
    rng = rng_of("other", cache, heads)
    spare = 300
    c = Cache(cache, lens, heads, seed=31, spare=spare)
    used = {int(x) for x in c.tables.flatten() if x >= 0}
    free = [b for b in range(c.blocks) if b not in used]
    rng.shuffle(free)
    for kind in ("any", "sorted"):
        counts = [0, 9, 1, 200, 2000]
        src = [[rng.randrange(n) for _ in range(m)] if n else [] for n, m in zip(lens, counts)]
        if kind == "sorted":
            src = [sorted(x) for x in src]
        start = [rng.randint(0, 40) for _ in lens]
        width = max((a + len(x) + 15) // 16 for a, x in zip(start, src)) + 1
        dst, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
        for s, (a, x) in enumerate(zip(start, src)):
            for b in range(a // 16, (a + len(x) + 15) // 16):
                dst[s, b] = free[at]
                at += 1
        check_moves(c, src, start, dst, pad=3)


@pytest.mark.parametrize("cache", CACHES)
def test_compaction_refuses_rows(cache):
    lens = [40, 40, 40]
    c = Cache(cache, lens, (2, 2, 64), seed=32)

    def call(src, start, cu, tables=None):
        before = pools_of(c)
        err = err_flag()
        compact_call(cache)(c.kp, c.vp, (c.tables if tables is None else tables).cuda(), i32(src), i32(start), i32(cu), err_flag=err)
        return before, pools_of(c), int(err)

    # rows from before their place, or from outside the table, stay; the others move
    before, after, err = call([5, 2, 20, 48, -1, 39], [3, 0, 0], [0, 6, 6, 6])
    assert err == pk.DEV_ERR_BAD_POS
    for was, now in zip(before, after):
        assert torch.equal(now, put(c, was, {(0, 3): (0, 5), (0, 5): (0, 20), (0, 8): (0, 39)}))
    before, after, err = call([30, 31, 32], [-1, 0, 48], [0, 1, 2, 3])
    assert err == pk.DEV_ERR_BAD_POS
    for was, now in zip(before, after):
        assert torch.equal(now, put(c, was, {(1, 0): (1, 31)}))
    # sequences whose rows leave the array
    for cu in ([0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 2, 9]):
        before, after, err = call([30, 31, 32], [0, 0, 0], cu)
        assert err & pk.DEV_ERR_BAD_CU
    # a block that is none
    for entry in (-1, c.blocks, -2**31):
        tables = c.tables.clone()
        tables[1, 2] = entry
        before, after, err = call([30, 31, 33, 32], [0, 0, 0], [0, 1, 3, 4], tables)
        assert err == pk.DEV_ERR_BAD_BLOCK
        for was, now in zip(before, after):
            assert torch.equal(now, put(c, was, {(0, 0): (0, 30), (1, 0): (1, 31), (2, 0): (2, 32)}))


def put(c, rows, moves):
    out = rows.clone()
    for (s, b), (_, p) in moves.items():
        out[int(c.tables[s, b // BLOCK]), b % BLOCK] = rows[int(c.tables[s, p // BLOCK]), p % BLOCK]
    return out


@pytest.mark.parametrize("cache", CACHES)
def test_compaction_in_a_graph(cache):
    c = Cache(cache, [300, 70], (2, 2, 128), seed=33)
    src, start, cu = i32([20, 40, 250, 9, 60]), i32([4, 1]), i32([0, 3, 5])
    tables = c.tables.cuda()
    keep = (c.kp.clone(), c.vp.clone())
    before = pools_of(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        compact_call(cache)(c.kp, c.vp, tables, src, start, cu)
    for was, t in zip(before, pools_of(c)):
        assert torch.equal(was, t)
    g.replay()
    for was, t in zip(before, pools_of(c)):
        assert torch.equal(moved(was, c.tables, c.tables, [[20, 40, 250], [9, 60]], [4, 1]), t)
    # the counts are the device's: fewer rows of other positions
    c.kp.copy_(keep[0])
    c.vp.copy_(keep[1])
    cu.copy_(i32([0, 0, 2]))
    src.copy_(i32([33, 50, -7, -7, -7]))
    g.replay()
    for was, t in zip(before, pools_of(c)):
        assert torch.equal(moved(was, c.tables, c.tables, [[], [33, 50]], [4, 1]), t)


# ---------------------------------------------------------------------------- a drafting step
@pytest.mark.parametrize("cache", CACHES)
def test_a_drafting_step(cache):
    # a tree is appended by its depths, attended, its accepted path moved up and the rest let go: the cache
    # is the one that plain appends of the path make
    heads, base, nodes = (8, 2, 128), 45, 20
    hq, hkv, d = heads
    rng = rng_of("step", cache)
    g = torch.Generator().manual_seed(40)
    wide = torch.float32 if cache == "f32" else torch.bfloat16
    bm = pk._native.BlockManager(64)
    a, b = bm.add_seq(), bm.add_seq()
    freq = frequencies(d)
    kp, vp = (pool_for(cache, 64, hkv, d) for _ in (0, 1))
    prompt = [torch.randn(base, h, d, generator=g).to(wide).cuda() for h in (hkv, hkv)]

    def table(s):
        return torch.tensor([bm.block_table(s, 16)], dtype=torch.int32, device="cuda")

    for s in (a, b):
        bm.prepare_append(s, 0, base)
        rope_call(cache)(kp, vp, None, None, *prompt, freq, table(s), i32([0]), i32([0, base]))
    parents = random_tree(nodes, rng)
    parents[0] = -1
    see = ancestors(parents)
    depth = [int(x) - 1 for x in see.sum(1)]
    leaf = max(range(nodes), key=lambda i: depth[i])
    path = [j for j in range(nodes) if see[leaf, j]]
    q, k, v = (torch.randn(nodes, h, d, generator=g).to(wide).cuda() for h in (hq, hkv, hkv))
    bm.prepare_append(a, base, nodes)
    turned, out, err = torch.empty_like(q), nan_like(q), err_flag()
    axes_call(cache)(kp, vp, turned, q, k, v, freq, None, i32([base + x for x in depth])[None], table(a), i32([base]), i32([0, nodes]),
                     err_flag=err)
    tree_call(cache)(out, turned, kp, vp, table(a), i32([base]), i32([0, nodes]), packed([see]).cuda(), d ** -0.5, nodes,
                     pk.tree_workspace(hq, hkv, d, nodes), err_flag=err)
    compact_call(cache)(kp, vp, table(a), i32([base + j for j in path]), i32([base]), i32([0, len(path)]), err_flag=err)
    bm.truncate(a, base + len(path))
    assert int(err) == 0 and bm.seq_len(a) == base + len(path)
    # the path alone, by plain appends
    at = torch.tensor(path, device="cuda")
    bm.prepare_append(b, base, len(path))
    alone = torch.empty(len(path), hq, d, dtype=wide, device="cuda")
    rope_call(cache)(kp, vp, alone, q[at].contiguous(), k[at].contiguous(), v[at].contiguous(), freq, table(b), i32([base]),
                     i32([0, len(path)]))
    assert torch.equal(alone, turned[at])
    n = base + len(path)
    for pool, keys in ((kp, True), (vp, False)):
        rows = unpacked(cache, pool, d, keys)
        one, two = (rows[torch.tensor(bm.block_table(s, (n + 15) // 16))].flatten(0, 1)[:n] for s in (a, b))
        assert torch.equal(one, two)
    # and what the tree's rows saw is what the path's rows see
    k64, v64 = (unpacked(cache, pool, d, keys)[torch.tensor(bm.block_table(b, (n + 15) // 16))].flatten(0, 1)[:n]
                for pool, keys in ((kp, True), (vp, False)))
    want, tol = attention(turned[at].cpu(), k64, v64, visible(base, torch.ones(len(path), len(path)).tril().bool()), d ** -0.5, cache, wide)
    within(out[at], want, tol)


# ---------------------------------------------------------------------------- the ends of the ranges
@pytest.mark.parametrize("cache", CACHES)
def test_more_sequences_than_threads(cache):
    rng = rng_of("1100", cache)
    ctx = [rng.randint(0, 40) for _ in range(1100)]
    counts = [rng.choice([0, 1, 1, 2]) for _ in ctx]
    sees = trees(counts, "1100", cache)
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (2, 1, 64), seed=40)
    q = c.queries(sum(counts))
    out = run_tree(c, ctx, sees, q, 0.125)
    check_tree(c, ctx, sees, q, 0.125, out)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_large_keys_and_small_queries(cache):
    # scores of ordinary size from factors that are not, in keys whose scales differ by 2^20
    ctx, counts, heads = [300], [9], (4, 2, 128)
    c = Cache(cache, [309], heads, seed=41)
    g = torch.Generator().manual_seed(42)
    k = (torch.randn(309, 2, 128, generator=g) * torch.exp2(100 + torch.linspace(0, 20, 309))[:, None, None]).to(torch.bfloat16)
    v = torch.randn(309, 2, 128, generator=g).to(torch.bfloat16)
    append = {"fp8": pk.append_kv_fp8, "fp4": pk.append_kv_fp4}.get(cache, pk.append_kv)
    append(c.kp, c.vp, k.cuda(), v.cuda(), c.tables.cuda(), i32([0]), i32([0, 309]))
    c.refresh()
    sees = trees(counts, "large")
    q = (c.queries(9).float() * 2.0 ** -120).to(torch.bfloat16)
    out = run_tree(c, ctx, sees, q, 0.1)
    check_tree(c, ctx, sees, q, 0.1, out)


@pytest.mark.parametrize("cache", CACHES)
def test_calls_at_once(cache):
    # two streams, each with a workspace of its own
    ctx, counts = [2500, 40, 700], [20, 3, 11]
    sees = trees(counts, "at once")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (8, 2, 64), seed=43)
    q = c.queries(sum(counts)).cuda()
    want = run_tree(c, ctx, sees, q, 0.1)
    rest = (c.tables.cuda(), i32(ctx), i32(cumulated(counts)), packed(sees).cuda(), 0.1, 20)
    runs = [(torch.cuda.Stream(), pk.tree_workspace(8, 2, 64, 20), nan_like(q)) for _ in (0, 1)]
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, ws, out in runs:
            with torch.cuda.stream(stream):
                tree_call(cache)(out, q, c.kp, c.vp, *rest, ws)
    torch.cuda.synchronize()
    for _, _, out in runs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
def test_outputs_on_a_16_byte_boundary(cache):
    ctx, counts = [130, 5], [7, 40]
    sees = trees(counts, "odd start")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], (6, 2, 64), seed=44)
    q = c.queries(47).cuda()
    e = 16 // q.element_size()
    room = torch.full((q.numel() + 2 * e,), 7.0, dtype=q.dtype, device="cuda")
    out = room[e:-e].view_as(q)
    assert out.data_ptr() % 32 == 16
    run_tree(c, ctx, sees, q, 0.1, out=out)
    check_tree(c, ctx, sees, q.cpu(), 0.1, out)
    assert bool((room[:e] == 7.0).all()) and bool((room[-e:] == 7.0).all())


@pytest.mark.parametrize("cache", CACHES)
def test_pools_past_32_bits(cache):
    # the sequences' blocks at both ends of pools of more than 4 GB
    ctx, counts, heads = [70, 200], [6, 17], (4, 2, 128)
    sees = trees(counts, "far blocks")
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=45)
    q = c.queries(23)
    each = c.kp[0].numel() * c.kp.element_size()
    blocks = 2**32 // each + 2 * c.blocks
    far = []
    for pool in (c.kp, c.vp):
        t = torch.empty((blocks,) + tuple(pool.shape[1:]), dtype=pool.dtype, device="cuda")
        t[-c.blocks:] = pool
        far.append(t)
    tables = torch.where(c.tables >= 0, c.tables + (blocks - c.blocks), -1).cuda()
    want, out = run_tree(c, ctx, sees, q, 0.1), nan_like(q.cuda())
    ws = pk.tree_workspace(4, 2, 128, 17)
    tree_call(cache)(out, q.cuda(), far[0], far[1], tables, i32(ctx), i32(cumulated(counts)), packed(sees).cuda(), 0.1, 17, ws)
    assert torch.equal(out, want)
    # kept rows to the first blocks, then in place at the far end
    src, start, cu = i32([69, 3, 40, 100, 215]), i32([0, 2]), i32([0, 3, 5])
    compact_call(cache)(far[0], far[1], tables, src, start, cu, dst_tables=i32([0, 1]).view(2, 1))
    compact_call(cache)(c.kp, c.vp, c.tables.cuda(), i32([3, 40, 69, 100, 215]), start, cu)
    compact_call(cache)(far[0], far[1], tables, i32([3, 40, 69, 100, 215]), start, cu)
    for pool, t in zip((c.kp, c.vp), far):
        assert torch.equal(pool.view(torch.uint8), t[-c.blocks:].view(torch.uint8))
    rows, near = (unpacked(cache, t, 128, True) for t in (far[0][-c.blocks:], far[0][:2]))
    first = c.tables[:, 0].tolist()
    assert torch.equal(near[0, 1], rows[first[0], 0]) and torch.equal(near[0, 2], rows[first[0], 1]) and torch.equal(near[0, 0], rows[first[0], 2])
    assert torch.equal(near[1, 2], rows[first[1], 2]) and torch.equal(near[1, 3], rows[first[1], 3])


@pytest.mark.parametrize("cache", CACHES)
def test_axes_in_a_graph(cache):
    # captured on a side stream, replayed over other positions, lengths and rows
    c = Cache(cache, [60, 90], (4, 2, 64), seed=46)
    x = torch.randn(20, 8, 64, generator=c.g).to(c.wide).cuda()
    q, k, v = torch.split(x, (4, 2, 2), dim=1)
    plane, places = i32([f % 3 for f in range(32)]), torch.randint(0, 5000, (3, 20), dtype=torch.int32, device="cuda")
    tables, start, cu = c.tables.cuda(), i32([50, 70]), i32([0, 8, 20])
    out = nan_like(q.contiguous())

    def call(kp, vp, o):
        axes_call(cache)(kp, vp, o, q, k, v, frequencies(64), plane, places, tables, start, cu)

    freq = frequencies(64)
    kp, vp = c.kp.clone(), c.vp.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        axes_call(cache)(kp, vp, out, q, k, v, freq, plane, places, tables, start, cu)
    for turn in range(2):
        places.random_(0, 9000)
        start.copy_(i32([50 - turn, 70 + turn]))
        x.normal_()
        kp.copy_(c.kp)
        vp.copy_(c.vp)
        kp2, vp2, out2 = c.kp.clone(), c.vp.clone(), nan_like(out)
        g.replay()
        call(kp2, vp2, out2)
        torch.cuda.synchronize()
        for a, b in ((kp, kp2), (vp, vp2), (out, out2)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
