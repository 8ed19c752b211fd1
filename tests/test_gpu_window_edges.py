"""The rotary append and the sliding-window attention where values leave the usual range, where
rows go by tiles, and where a sequence's parts do not divide evenly (tolerances: see
_window_common.py, and beside each test what it adds)."""
import math
import re
import warnings

import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _window_common import (BLOCK, Cache, attention, half_step, nan_like, pool_for, rope_call, rotated, visible, within)
from test_gpu_window import cu_of, err_flag, frequencies, i32, place, rope_inputs, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def refill(c, k, v):
    """Other rows [tokens][Hkv][D] into the cache, in the order of the sequences."""
    append = {"fp8": pk.append_kv_fp8, "fp4": pk.append_kv_fp4}.get(c.cache, pk.append_kv)
    append(c.kp, c.vp, k.to(c.wide).cuda(), v.to(c.wide).cuda(), c.tables.cuda(), i32([0] * len(c.lens)), i32(c.cu))
    c.refresh()


def check_range(c, q, window, sinks, scale, out):
    """Outputs of the 8- and 4-bit caches with a tolerance that follows the values.

    A probability times its value's scale is brought to f16 by a power of two that takes the
    largest scale so far to between 2^11 and 2^15, so what rounds below f16's normal range is off
    by at most 2^-25 of that unit: 2^-36 of the largest scale, times the largest code at most
    2^-36 max |v| for each key."""
    for s, n in enumerate(c.lens):
        see = visible(torch.tensor([n - 1]), n, window, sinks)
        want, tol = attention(q[s:s + 1], c.k[s], c.v[s], see, scale, "f16", q.dtype)
        G = c.hq // c.hkv
        for h in range(c.hkv):
            tol[:, h * G:(h + 1) * G] += n * 2.0 ** -36 * float(c.v[s][see[0], h].abs().max())
        within(out[s:s + 1], want, tol, f"sequence {s} of length {n}")


# ---------------------------------------------------------------------------- decode: values
def sizes(kind, n, hkv, g):
    """Factors of the value rows [tokens][Hkv][1]."""
    if kind == "mixed":                # from row to row, eleven orders of magnitude
        return 10.0 ** (torch.rand(n, hkv, 1, generator=g) * 11 - 5.5)
    if kind == "rising":               # raised again and again, within a part and from part to part
        return torch.logspace(-20, 20, n).view(n, 1, 1).expand(n, hkv, 1)
    if kind == "falling":
        return torch.logspace(20, -20, n).view(n, 1, 1).expand(n, hkv, 1)
    return torch.full((n, hkv, 1), float(kind))


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64)])
@pytest.mark.parametrize("kind", ["1e-20", "1e-5", "1e-2", "1", "2e5", "1e30", "mixed", "rising", "falling"])
def test_decode_of_values_of_any_size(cache, heads, kind):
    lens = [1, 40, 700, 2600]
    c = Cache(cache, lens, heads, seed=51)
    g = torch.Generator().manual_seed(52)
    n = sum(lens)
    refill(c, torch.randn(n, heads[1], heads[2], generator=g),
           torch.randn(n, heads[1], heads[2], generator=g) * sizes(kind, n, heads[1], g))
    q = c.queries(len(lens))
    for window, sinks in ((2500, 4), (33, 0)):
        check_range(c, q, window, sinks, 0.1, run_decode(c, lens, q, window, sinks, 0.1))


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
@pytest.mark.parametrize("kind", ["mixed", "rising", "falling"])
def test_decode_of_values_of_any_size_is_the_same_in_every_batch(cache, kind):
    # (every part starts with a reference of its own, whatever CTA does it)
    lens, heads = [2300, 900], (32, 8, 128)
    c = Cache(cache, lens, heads, seed=58)
    g = torch.Generator().manual_seed(59)
    refill(c, torch.randn(3200, 8, 128, generator=g), torch.randn(3200, 8, 128, generator=g) * sizes(kind, 3200, 8, g))
    q = c.queries(2)
    out = run_decode(c, lens, q, 2040, 20, 0.1)
    for n in (1, 3, 8, 16, 40, 160):
        at = torch.arange(n) % 2
        many = run_decode(c, [lens[i] for i in at], q[at], 2040, 20, 0.1, tables=c.tables[at])
        assert torch.equal(many, out[at.cuda()]), n


def small_values_beside_a_hidden_weight(cache, d, small):
    # the first key has the largest value and no weight (a score 60 or more below the others'): what the
    # others' probabilities lose beside its scale stays within the tolerance
    lens, heads = [4], (2, 2, d)
    c = Cache(cache, lens, heads, seed=54)
    g = torch.Generator().manual_seed(d - round(math.log2(small)))
    q = torch.randn(1, 2, d, generator=g).to(c.wide)
    k, v = torch.randn(4, 2, d, generator=g), torch.randn(4, 2, d, generator=g)
    k[0] = -8 * q[0].float()
    v[1:] *= small
    refill(c, k, v)
    check_range(c, q, 100, 0, d ** -0.5, run_decode(c, lens, q, 100, 0, d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small", [2.0 ** -22, 2.0 ** -26, 2.0 ** -30])
def test_fp8_decode_of_small_values_beside_a_hidden_weight(d, small):
    small_values_beside_a_hidden_weight("fp8", d, small)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small", [2.0 ** -22, 2.0 ** -26, 2.0 ** -30])
def test_fp4_decode_of_small_values_beside_a_hidden_weight(d, small):
    small_values_beside_a_hidden_weight("fp4", d, small)


# ---------------------------------------------------------------------------- decode: queries
@pytest.mark.parametrize("cache", ["fp8", "fp4"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64)])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 7e4, 1e30])
def test_decode_of_queries_of_any_size(cache, heads, size):
    lens = [20, 700]
    c = Cache(cache, lens, heads, seed=53)
    q = (c.queries(2).float() * size).to(c.wide)
    check_range(c, q, 600, 4, 0.1 / size, run_decode(c, lens, q, 600, 4, 0.1 / size))
    # heads of one group apart by fourteen orders of magnitude; and a head of zeros
    q = c.queries(2).float()
    q[:, 0] *= 1e7
    q[:, 1] *= 1e-7
    q[:, 2] = 0
    q = q.to(c.wide)
    for scale in (1e-8, 1e6):
        # (scores beyond fp32's exponent of the others are still finite: the weights of a few keys)
        check_range(c, q, 600, 4, scale, run_decode(c, lens, q, 600, 4, scale))


# ---------------------------------------------------------------------------- decode: f32
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128)])
def test_f32_decode_of_infinities_and_the_largest_values(heads):
    hq, hkv, d = heads
    lens = [200, 1, 900]
    c = Cache("f32", lens, heads, seed=55)
    k, v = (torch.cat(x).float() for x in (c.k, c.v))
    last = torch.finfo(torch.float32).max
    # keys that score -inf get weight 0, also as the first ones of a warp's walk
    away = list(range(64)) + [100, 199]
    k[away, :, 0] = float("-inf")
    # a value that is not finite reaches its dim alone; the largest one stays what it is
    v[120, :, 5] = float("inf")
    v[200, :, 7] = last
    # the largest keys, and queries that bring them back
    k[201 + 50, :, 3] = last
    refill(c, k, v)
    q = torch.rand(3, hq, d, generator=c.g) + 0.1
    q[2, :, 3] = 8.0 / last
    out = run_decode(c, lens, q, 1000, 0, 0.125).cpu()
    assert bool((out[0, :, 5] == float("inf")).all())
    out[0, :, 5] = 0
    c.k[0][away], c.v[0][120, :, 5] = 0, 0
    for s, n in enumerate(lens):
        see = torch.ones(1, n, dtype=torch.bool)
        if s == 0:
            see[0, away] = False
        want, tol = attention(q[s:s + 1], c.k[s], c.v[s], see, 0.125, "f32", q.dtype)
        if s == 0:
            want[:, :, 5] = 0
        within(out[s:s + 1], want, tol, f"sequence {s}")
    # a part that is done again gives the same bits in batches of every size
    for n in (1, 2, 8, 30, 200):
        at = torch.arange(n) % 3
        many = run_decode(c, [lens[i] for i in at], q[at], 1000, 0, 0.125, tables=c.tables[at])
        many[at.cuda() == 0, :, 5] = 0
        assert torch.equal(many, out.cuda()[at.cuda()]), n


# ---------------------------------------------------------------------------- prefill
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(1000, 0), (70, 4), (300, 140)])
def test_prefill_of_keys_that_score_minus_infinity(heads, window, sinks):
    # weight 0, whole tiles of them among others and before a row's first key; rows that see no other key give zeros
    starts, counts = [0, 300], [200, 260]
    c = Cache("bf16", [200, 560], heads, seed=56)
    q = (torch.rand(460, heads[0], heads[2], generator=c.g) + 0.05).to(c.wide)
    away = [list(range(64)) + [100, 199], list(range(128, 300)) + [310, 420]]
    for s in (0, 1):
        for t in away[s]:
            c.kp[int(c.tables[s, t // BLOCK]), :, :, t % BLOCK, 0] = float("-inf")
    out = run_prefill(c, starts, counts, q, window, sinks, 0.125)
    for s, (a, n, row) in enumerate(zip(starts, counts, (0, 200))):
        see = visible(a + torch.arange(n), a + n, window, sinks)
        see[:, away[s]] = False
        k = c.k[s].clone()
        k[away[s]] = 0
        want, tol = attention(q[row:row + n], k, c.v[s], see, 0.125, "bf16", q.dtype)
        within(out[row:row + n], want, tol, f"sequence {s}")


# ---------------------------------------------------------------------------- decode: parts
@pytest.mark.parametrize("cache,heads,windows", [
    ("bf16", (32, 8, 128), (2276, 2150)),                # 7 and 6 parts
    ("bf16", (14, 2, 64), (2276, 1250)),                 # 5 and 3
    ("fp8", (32, 8, 128), (2276, 2150)),
    ("fp8", (14, 2, 64), (2600,)),                       # 6
    ("fp4", (32, 8, 128), (4300,)),                      # 7
    ("f32", (12, 12, 64), (2276, 4300, 4600, 5400)),     # 7, 12, 13 and 15
    ("f32", (15, 3, 128), (2276,)),                      # 7
])
def test_decode_is_the_same_where_parts_do_not_divide_evenly(cache, heads, windows):
    lens = [6300, 2290, 4700, 17]
    c = Cache(cache, lens, heads, seed=57)
    q = c.queries(len(lens))
    for window in windows:
        out = run_decode(c, lens, q, window, 4, 0.1)
        for s, n in enumerate(lens):
            want, tol = attention(q[s:s + 1], c.k[s], c.v[s], visible(torch.tensor([n - 1]), n, window, 4), 0.1, cache, q.dtype)
            within(out[s:s + 1], want, tol, f"sequence {s} of length {n}")
        for n in (1, 2, 3, 5, 8, 12, 16, 24, 40, 75, 160):
            at = torch.arange(n) % len(lens)
            many = run_decode(c, [lens[i] for i in at], q[at], window, 4, 0.1, tables=c.tables[at])
            assert torch.equal(many, out[at.cuda()]), (window, n)


# ---------------------------------------------------------------------------- rotary append
def captured(call, tmp_path):
    """What the runtime says of the kernels that `call` launches."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    at = tmp_path / "graph.dot"
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        graph.debug_dump(str(at))
    return at.read_text()


def kernels_of(call, tmp_path):
    """The rotary append's kernels that `call` launches, by name."""
    text = captured(call, tmp_path)
    return {name for name in ("rope_append_kernel", "rope_append_tile_kernel") if name in text}


CACHES = ["bf16", "f32", "fp8", "fp4"]


def test_rope_append_goes_by_rows_and_by_tiles(tmp_path):
    for cache in CACHES:
        most = 512 if cache in ("bf16", "f32") else 256
        for counts, want in (([most], "rope_append_kernel"), ([most + 1], "rope_append_tile_kernel"),
                             ([8] * 200, "rope_append_kernel"), ([40] * 20, "rope_append_tile_kernel")):
            _, (dq, dk, dv) = rope_inputs(cache, counts, (4, 2, 64), False, seed=1)
            tables, _, _, blocks = place([3] * len(counts), counts)
            args = (pool_for(cache, blocks, 2, 64), pool_for(cache, blocks, 2, 64), nan_like(dq), dq, dk, dv, frequencies(64),
                    tables.cuda(), i32([3] * len(counts)), cu_of(counts))
            assert kernels_of(lambda: rope_call(cache)(*args), tmp_path) == {want}, (cache, counts[0])


@pytest.mark.parametrize("cache,threads", [("bf16", 128), ("fp8", 128), ("f32", 256)])
def test_rope_append_shares_tiles_as_the_gpu_has_room(cache, threads, tmp_path):
    # 154 tiles in as many shares as 520 threads for each SM allow
    n, (hq, hkv, d) = 154 * BLOCK, (32, 8, 128)
    _, (dq, dk, dv) = rope_inputs(cache, [n], (hq, hkv, d), False, seed=64)
    tables = torch.arange(154, dtype=torch.int32).view(1, 154).cuda()
    args = (pool_for(cache, 154, hkv, d), pool_for(cache, 154, hkv, d), nan_like(dq), dq, dk, dv, frequencies(d), tables,
            i32([0]), cu_of([n]))
    # (a grid of one share has one dimension)
    grid = re.search(r"rope_append_tile_kernel\S*?<\\<(?:\\\{\d+,(\d+)\\\}|\d+),(\d+)", captured(lambda: rope_call(cache)(*args), tmp_path))
    shares, room = int(grid[1] or 1), torch.cuda.get_device_properties(0).multi_processor_count * 520 // threads
    assert int(grid[2]) == threads and shares == max(1, room // 154)


# 712 rows of six sequences, 32 and more on average: tiles for every type of pool
TILE_COUNTS, TILE_STARTS = [160, 33, 0, 250, 200, 69], [0, 5, 9, 50, 31, 130]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 3, 128), (26, 1, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_of_tiles_in_place_and_without_queries(cache, heads, interleaved, tmp_path):
    hq, hkv, d = heads
    (q, k, v), (dq, dk, dv) = rope_inputs(cache, TILE_COUNTS, heads, True, seed=61)
    tables, pos, blk, blocks = place(TILE_STARTS, TILE_COUNTS)
    freq = frequencies(d)
    args = (freq, tables.cuda(), i32(TILE_STARTS), cu_of(TILE_COUNTS), interleaved)
    pools = [[pool_for(cache, blocks, hkv, d) for _ in (0, 1)] for _ in range(3)]
    out = nan_like(dq.contiguous())
    assert kernels_of(lambda: rope_call(cache)(*pools[0], out, dq, dk, dv, *args), tmp_path) == {"rope_append_tile_kernel"}
    rope_call(cache)(*pools[0], out, dq, dk, dv, *args)
    rope_call(cache)(*pools[1], None, None, dk, dv, *args)
    rope_call(cache)(*pools[2], dq, dq, dk, dv, *args)             # queries turned where they are
    want, size = rotated(q, pos, freq.cpu(), interleaved)
    within(out, want, half_step(q.dtype) * want.abs() + 5e-7 * size + 1e-30, "queries")
    assert torch.equal(dq, out)
    for a in pools[1:]:
        for x, y in zip(a, pools[0]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# prefix sums over the 712 rows: a wrong end, backwards, negative, past the rows, not from 0
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("cu", [[0, 160, 193, 193, 443, 643, 700], [0, 160, 193, 193, 443, 643, 800],
                                [0, 193, 160, 193, 443, 643, 712], [0, -40, 193, 193, 443, 643, 712],
                                [0, 160, 193, 193, 900, 643, 712], [16, 160, 193, 193, 443, 643, 712],
                                [0, 2**31 - 1, -2**31, 193, 443, 643, 712], [712, 643, 443, 193, 193, 160, 0]])
def test_rope_append_of_tiles_flags_bad_prefix_sums(cache, cu, tmp_path):
    heads = (4, 2, 64)
    (q, k, v), (dq, dk, dv) = rope_inputs(cache, TILE_COUNTS, heads, True, seed=62)
    tables = torch.arange(6 * 24, dtype=torch.int32).view(6, 24)
    freq, starts = frequencies(64), TILE_STARTS
    kp, vp = pool_for(cache, 6 * 24, 2, 64), pool_for(cache, 6 * 24, 2, 64)
    out, err = nan_like(dq.contiguous()), err_flag()
    args = (freq, tables.cuda(), i32(starts), i32(cu))
    call = lambda: rope_call(cache)(kp, vp, out, dq, dk, dv, *args, err_flag=err)
    assert kernels_of(call, tmp_path) == {"rope_append_tile_kernel"}
    call()
    assert int(err) & pk.DEV_ERR_BAD_CU
    # every row that lies in one sequence alone, one within the rows, is turned by its place there
    claims = torch.zeros(712, dtype=torch.int64)
    at = torch.zeros(712, dtype=torch.int64)
    for s in range(6):
        a, b = cu[s], cu[s + 1]
        if 0 <= a <= b <= 712:
            claims[a:b] += 1
            at[a:b] = starts[s] + torch.arange(b - a)
    rising = all(a <= b for a, b in zip(cu, cu[1:]))
    done = ~out.isnan().any(-1).any(-1).cpu()
    assert not bool(done[claims == 0].any())
    ok = (claims == 1) & (at < 24 * BLOCK)
    if rising:
        assert torch.equal(done, ok)
    else:
        ok &= done                                        # (the search may miss sequences of sums that fall)
    want, size = rotated(q, at, freq.cpu(), False)
    within(out[ok.cuda()], want[ok], (half_step(q.dtype) * want.abs() + 5e-7 * size + 1e-30)[ok], "queries")


@pytest.mark.parametrize("d", [64, 128])
def test_rope_append_fp8_keeps_the_sign_of_zeros(d):
    # values are never turned: the plain append's bytes, -0 among them, row by row and by tiles
    g = torch.Generator().manual_seed(63)
    n, hkv = 1200, 2
    v = torch.randn(n, hkv, d, generator=g)
    v[torch.rand(n, hkv, d, generator=g) < 0.1] = -0.0
    v[torch.rand(n, hkv, d, generator=g) < 0.1] = 0.0
    dk, dv = (torch.randn(n, hkv, d, generator=g).bfloat16().cuda(), v.bfloat16().cuda())
    for counts in ([1] * n, [n]):
        blocks = sum((x + BLOCK - 1) // BLOCK for x in counts)
        tables = torch.arange(blocks, dtype=torch.int32).view(len(counts), -1).cuda()
        starts, cu = i32([0] * len(counts)), cu_of(counts)
        pools = [[pool_for("fp8", blocks, hkv, d) for _ in (0, 1)] for _ in (0, 1)]
        pk.rope_append_kv_fp8(*pools[0], None, None, dk, dv, frequencies(d), tables, starts, cu)
        pk.append_kv_fp8(*pools[1], dk, dv, tables, starts, cu)
        assert bool((pools[1][1][..., :BLOCK * d] == 0x80).any()) and torch.equal(pools[0][1], pools[1][1])


def test_bounds_far_below_are_refused_both_ways():
    c = Cache("bf16", [40], (4, 2, 64), seed=65)
    q = c.queries(1).cuda()
    call = lambda w, n, **kw: pk.decode_attention_window(torch.empty_like(q), q, c.kp, c.vp, c.tables.cuda(), i32([40]), 0.1, w, n, **kw)
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        for w, n in ((-2**32 + 5, 0), (-2**63, 0), (5, -2**32 + 1), (-2**100, 3)):
            with pytest.raises(pk.PagedKVError):
                call(w, n, **kw)
        call(2**32 + 5, 2**33, **kw)
