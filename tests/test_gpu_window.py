"""The rotary append and the sliding-window attention against a plain 64-bit implementation
(tests/_window_common.py, which derives the tolerances)."""
import os
import subprocess
import sys

import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _window_common import (BLOCK, Cache, attention, decode_call, half_step, nan_like, pool_for, rope_call,
                            rotated, unpacked, visible, within)

pytestmark = pytest.mark.gpu

HEADS = [(4, 4, 64), (14, 2, 64), (8, 1, 128), (8, 2, 128), (9, 3, 128)]
CACHES = ["bf16", "f32", "fp8", "fp4"]


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def err_flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def frequencies(rotary, base=10000.0):
    return (base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).cuda()


# ---------------------------------------------------------------------------- decode
def run_decode(c, lens, q, window, sinks, scale, tables=None, err=None):
    out = nan_like(q.cuda())
    decode_call(c.cache)(out, q.cuda(), c.kp, c.vp, (c.tables if tables is None else tables).cuda(), i32(lens), scale,
                         window, sinks, err_flag=err)
    return out


def check_decode(c, lens, q, window, sinks, scale, out):
    for s, n in enumerate(lens):
        want, tol = attention(q[s:s + 1], c.k[s][:n], c.v[s][:n], visible(torch.tensor([n - 1]), n, window, sinks), scale,
                              c.cache, q.dtype)
        within(out[s:s + 1], want, tol, f"sequence {s} of length {n}")


LENS = [0, 1, 15, 16, 17, 33, 100, 257]
WINDOWS = [(1, 0), (1, 1), (16, 0), (17, 4), (40, 16), (33, 70), (100, 17), (10**9, 0), (2**40, 3)]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", HEADS)
def test_decode_sees_the_window_and_the_sinks_only(cache, heads):
    # every hidden slot holds NaN, blocks without a visible slot are gone from the table
    for window, sinks in WINDOWS:
        c = Cache(cache, LENS, heads, seed=window % 1000 + sinks)
        for s, n in enumerate(LENS):
            keep = visible(torch.tensor([n - 1]), n, window, sinks)[0] if n else torch.zeros(0, dtype=torch.bool)
            c.poison(s, keep)
        q = c.queries(len(LENS))
        err = err_flag()
        out = run_decode(c, LENS, q, window, sinks, heads[2] ** -0.5, err=err)
        assert int(err) == 0
        assert bool((out[0] == 0).all())                       # an empty context
        check_decode(c, LENS, q, window, sinks, heads[2] ** -0.5, out)


@pytest.mark.parametrize("cache", CACHES)
def test_decode_over_many_partitions(cache):
    lens = [3000, 1, 2049, 1500, 2600]
    c = Cache(cache, lens, (8, 2, 128), seed=3)
    q = c.queries(len(lens))
    for window, sinks in ((2048, 4), (1000, 33), (2500, 0), (10**6, 0)):
        out = run_decode(c, lens, q, window, sinks, 0.1)
        check_decode(c, lens, q, window, sinks, 0.1, out)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(8, 1, 128), (8, 8, 64)])
def test_decode_over_the_most_partitions(cache, heads):
    # a window that takes the largest cluster, in one and in many CTAs (the same bits)
    n, window = 12500, 12000
    c = Cache(cache, [n], heads, seed=12)
    q = c.queries(1)
    alone = run_decode(c, [n], q, window, 20, 0.1)
    check_decode(c, [n], q, window, 20, 0.1, alone)
    many = 80
    out = nan_like(q.repeat(many, 1, 1).cuda())
    decode_call(cache)(out, q.repeat(many, 1, 1).cuda(), c.kp, c.vp, c.tables.repeat(many, 1).cuda(), i32([n] * many), 0.1,
                       window, 20)
    assert bool((out == alone).all())


@pytest.mark.parametrize("cache", CACHES)
def test_decode_on_two_streams_and_in_two_graphs_at_once(cache):
    lens = [1500, 700]
    c = Cache(cache, lens, (8, 2, 128), seed=13)
    q, other = c.queries(2), c.queries(2)
    want = [run_decode(c, lens, x, 1024, 4, 0.1) for x in (q, other)]
    args = (c.kp, c.vp, c.tables.cuda(), i32(lens), 0.1, 1024, 4)
    outs, qs = [nan_like(w) for w in want], [q.cuda(), other.cuda()]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for x, o, s in zip(qs, outs, streams):
        with torch.cuda.stream(s):
            for _ in range(20):
                decode_call(cache)(o, x, *args)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for x, o, g in zip(qs, outs, graphs):
        o.fill_(float("nan"))
        with torch.cuda.graph(g):
            decode_call(cache)(o, x, *args)
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


FIRST_IN_A_CAPTURE = """
import sys, torch
sys.path.insert(0, "tests")
import paged_kv_cache_207_gb300 as pk
from _window_common import Cache, nan_like
c = Cache("bf16", [2000, 700], (8, 2, 128), seed=3)
q, lens = c.queries(2).cuda(), torch.tensor([2000, 700], dtype=torch.int32, device="cuda")
kn, vn = torch.randn(2, 2, 2, 128, device="cuda").bfloat16()
start, cu = lens - 1, torch.arange(3, dtype=torch.int32, device="cuda")
freq = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
tables, out, turned = c.tables.cuda(), nan_like(q), torch.empty_like(q)
def step():
    pk.rope_append_kv(c.kp, c.vp, turned, q, kn, vn, freq, tables, start, cu)
    pk.decode_attention_window(out, turned, c.kp, c.vp, tables, lens, 0.1, 1500, 4)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = out.clone()
out.fill_(float("nan"))
step()
torch.cuda.synchronize()
assert torch.equal(out, got) and not bool(got.isnan().any())
"""


def test_first_call_of_a_process_is_captured():
    # (what the library asks the runtime once, clusters' room among it, is asked within the capture)
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("cache", CACHES)
def test_decode_batched_equals_alone_and_repeats(cache):
    lens = [700, 5, 1300, 64, 0, 2000]
    c = Cache(cache, lens, (14, 2, 64), seed=5)
    q = c.queries(len(lens))
    out = run_decode(c, lens, q, 600, 20, 0.125)
    for _ in range(5):
        assert torch.equal(run_decode(c, lens, q, 600, 20, 0.125), out)
    for s in range(len(lens)):
        one = run_decode(c, lens[s:s + 1], q[s:s + 1], 600, 20, 0.125, tables=c.tables[s:s + 1])
        assert torch.equal(one[0], out[s])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(32, 8, 128), (15, 3, 128), (14, 2, 64)])
def test_decode_is_the_same_in_batches_of_every_size(cache, heads):
    # (a CTA takes one, two, four or all of a sequence's parts, as the batch grows)
    lens = [2300, 2020, 900, 1300, 17, 0]
    c = Cache(cache, lens, heads, seed=31)
    q = c.queries(len(lens))
    out = run_decode(c, lens, q, 2040, 20, 0.1)
    check_decode(c, lens, q, 2040, 20, 0.1, out)
    for n in (1, 2, 3, 5, 8, 12, 16, 24, 40, 75, 160):
        at = torch.arange(n) % len(lens)
        many = run_decode(c, [lens[i] for i in at], q[at], 2040, 20, 0.1, tables=c.tables[at])
        assert torch.equal(many, out[at.cuda()]), n


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 8.0])
def test_decode_scales(cache, scale):
    lens = [90, 33]
    c = Cache(cache, lens, (8, 2, 128), seed=7)
    q = c.queries(2)
    check_decode(c, lens, q, 50, 4, scale, run_decode(c, lens, q, 50, 4, scale))


def test_decode_window_over_everything_agrees_with_the_full_decode():
    lens = [500, 31, 1000]
    c = Cache("bf16", lens, (8, 2, 128), seed=8)
    q = c.queries(3)
    out = run_decode(c, lens, q, 1000, 0, 0.1)
    full = torch.empty_like(out)
    pk.decode_attention(full, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(lens), 0.1,
                        workspace=pk.decode_workspace(3, 8, 2, 128, c.width))
    for s, n in enumerate(lens):
        want, tol = attention(q[s:s + 1], c.k[s], c.v[s], visible(torch.tensor([n - 1]), n, 10**6, 0), 0.1,
                              "bf16", q.dtype)
        within(out[s:s + 1], want, tol)
        within(full[s:s + 1], want, tol)


@pytest.mark.parametrize("cache", ["bf16"])
def test_decode_scores_of_minus_infinity(cache):
    # visible keys that score -inf get weight 0, also as the first ones of a warp's walk
    lens = [200]
    c = Cache(cache, lens, (4, 4, 64), seed=9)
    q = torch.ones(1, 4, 64).to(c.wide)
    for t in list(range(0, 64)) + [100, 199]:
        c.kp[int(c.tables[0, t // 16]), :, :, t % 16, 0] = float("-inf")
    out = run_decode(c, lens, q, 200, 0, 0.125)
    see = torch.ones(1, 200, dtype=torch.bool)
    see[0, :64] = False
    see[0, 100] = see[0, 199] = False
    want, tol = attention(q, c.k[0], c.v[0], see, 0.125, cache, q.dtype)
    within(out, want, tol)


@pytest.mark.parametrize("cache", CACHES)
def test_decode_flags_bad_data_and_an_earlier_abort(cache):
    lens = [100, 100]
    c = Cache(cache, lens, (8, 2, 128), seed=11)
    q = c.queries(2)
    good = run_decode(c, lens, q, 30, 4, 0.1)
    tables = c.tables.clone()
    tables[0, 3] = c.blocks                        # hidden: never read
    err = err_flag()
    assert torch.equal(run_decode(c, lens, q, 30, 4, 0.1, tables=tables, err=err), good) and int(err) == 0
    tables[0, 5] = c.blocks                        # in the window
    out = run_decode(c, lens, q, 30, 4, 0.1, tables=tables, err=err)
    assert int(err) == pk.DEV_ERR_BAD_BLOCK and torch.equal(out[1], good[1])
    err.zero_()
    run_decode(c, [100, c.width * BLOCK + 1], q, 30, 4, 0.1, err=err)
    assert int(err) & pk.DEV_ERR_BAD_POS
    err.fill_(pk.DEV_ERR_TIMEOUT)
    assert bool(run_decode(c, lens, q, 30, 4, 0.1, err=err).isnan().all())
    assert int(err) == pk.DEV_ERR_TIMEOUT
    err.zero_()
    assert torch.equal(run_decode(c, lens, q, 30, 4, 0.1, err=err), good)


# ---------------------------------------------------------------------------- rotary append
def rope_inputs(cache, counts, heads, fused, seed):
    hq, hkv, d = heads
    g = torch.Generator().manual_seed(seed)
    n = sum(counts)
    wide = torch.float32 if cache == "f32" else torch.bfloat16
    x = torch.randn(n, hq + 2 * hkv, d, generator=g).to(wide)
    parts = torch.split(x, (hq, hkv, hkv), 1)
    dev = torch.split(x.cuda(), (hq, hkv, hkv), 1) if fused else [p.contiguous().cuda() for p in parts]
    return parts, dev


def place(starts, counts, width=None):
    """Tables with blocks for the new rows only, and each row's position, block and slot."""
    width = width or max(1, max((s + n + BLOCK - 1) // BLOCK for s, n in zip(starts, counts)))
    tables = torch.full((len(starts), width), -1, dtype=torch.int32)
    used, pos, blk = 0, [], []
    for s, (a, n) in enumerate(zip(starts, counts)):
        for p in range(a, a + n):
            if tables[s, p // BLOCK] < 0:
                tables[s, p // BLOCK] = used
                used += 1
            pos.append(p)
            blk.append(int(tables[s, p // BLOCK]))
    perm = torch.randperm(used + 2, generator=torch.Generator().manual_seed(used))
    tables = torch.where(tables >= 0, perm[tables.clamp(min=0).long()].int(), -1).int()
    return tables, torch.tensor(pos, dtype=torch.int64), perm[torch.tensor(blk, dtype=torch.int64)], used + 2


def cu_of(counts):
    return i32([sum(counts[:i]) for i in range(len(counts) + 1)])


ROPE_SHAPES = [
    # starts, counts: decode rows, ragged chunks with an empty one, a block's edges, far positions
    ([5, 16, 131071, 2000003, 0], [1, 1, 1, 1, 1]),
    ([0, 14, 700000, 31], [40, 3, 0, 17]),
    ([15], [1]),
]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads,rotary", [((4, 2, 64), 64), ((14, 2, 64), 48), ((8, 2, 128), 128), ((9, 3, 128), 32),
                                          ((3, 1, 128), 112), ((2, 2, 64), 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_rotates_and_stores(cache, heads, rotary, interleaved):
    hq, hkv, d = heads
    freq = frequencies(rotary)
    for n, (starts, counts) in enumerate(ROPE_SHAPES):
        fused = n == 1
        (q, k, v), (dq, dk, dv) = rope_inputs(cache, counts, heads, fused, seed=n)
        tables, pos, blk, blocks = place(starts, counts)
        kp, vp = pool_for(cache, blocks, hkv, d), pool_for(cache, blocks, hkv, d)
        before = kp.clone(), vp.clone()
        out, err = nan_like(dq.contiguous()), err_flag()
        rope_call(cache)(kp, vp, out, dq, dk, dv, freq, tables.cuda(), i32(starts), cu_of(counts), interleaved, err_flag=err)
        assert int(err) == 0
        want, size = rotated(q, pos, freq.cpu(), interleaved)
        within(out, want, half_step(q.dtype) * want.abs() + 5e-7 * size + 1e-30, "queries")
        want, size = rotated(k, pos, freq.cpu(), interleaved)
        slot = pos % BLOCK
        got_k, got_v = unpacked(cache, kp, d, True)[blk, slot], unpacked(cache, vp, d, False)[blk, slot]
        if cache in ("bf16", "f32"):
            within(got_k, want, half_step(k.dtype) * want.abs() + 5e-7 * size + 1e-30, "keys")
            assert torch.equal(got_v, v.double())
        elif cache == "fp8":
            # half a step of E4M3: 2^-4 of the value, 2^-10 scales below its normal range
            unit = want.abs().amax(-1, keepdim=True) / 448
            within(got_k, want, torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit) + 1e-5 * unit * 448, "keys")
        else:
            # half a step of E2M1 at the block's scale; above 6 scales the code saturates
            x = want.unflatten(-1, (d // 32, 32))
            top = x.abs().amax(-1, keepdim=True)
            unit = 2.0 ** (torch.floor(torch.log2(top)) - 2)
            y = x.abs() / unit
            step = torch.where(y < 2, 0.25, torch.where(y < 4, 0.5, torch.where(y <= 7, 1.0, y - 6)))
            edge = (torch.log2(top * (1 + 1e-5)).floor() != torch.log2(top * (1 - 1e-5)).floor())
            # a scale may go either way there: unrotated bf16 values hit a power of two in one of
            # 128 blocks, so a few blocks at most
            assert int(edge.sum()) <= 2 + edge.numel() // 32
            within(got_k, want, (step * unit + 1e-5 * top + torch.where(edge, top, 0.0)).flatten(-2), "keys")
        if cache in ("fp8", "fp4"):
            # values are stored as the plain append stores them, byte for byte
            k2, v2 = before[0].clone(), before[1].clone()
            (pk.append_kv_fp8 if cache == "fp8" else pk.append_kv_fp4)(
                k2, v2, dk.contiguous(), dv.contiguous(), tables.cuda(), i32(starts), cu_of(counts))
            assert torch.equal(v2, vp)
        # nothing but the rows' slots changed
        hit = torch.zeros(blocks, BLOCK, dtype=torch.bool)
        hit[blk, slot] = True
        for pool, old, keys in ((kp, before[0], True), (vp, before[1], False)):
            same = unpacked(cache, pool, d, keys) == unpacked(cache, old, d, keys)
            assert bool(same[~hit].all())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_at_position_zero_is_the_plain_append(cache, interleaved):
    heads, counts = (8, 2, 128), [1] * 6
    (q, k, v), (dq, dk, dv) = rope_inputs(cache, counts, heads, False, seed=2)
    tables = torch.randperm(8)[:6].int().view(6, 1).cuda()
    pools = [[pool_for(cache, 8, 2, 128) for _ in (0, 1)] for _ in (0, 1)]
    out = nan_like(dq)
    rope_call(cache)(*pools[0], out, dq, dk, dv, frequencies(128), tables, i32([0] * 6), cu_of(counts), interleaved)
    plain = {"fp8": pk.append_kv_fp8, "fp4": pk.append_kv_fp4}.get(cache, pk.append_kv)
    plain(*pools[1], dk, dv, tables, i32([0] * 6), cu_of(counts))
    assert torch.equal(out, dq)
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])


def test_rope_append_in_place_and_without_queries():
    heads, counts, starts = (8, 2, 128), [3, 20], [100, 7]
    (q, k, v), (dq, dk, dv) = rope_inputs("bf16", counts, heads, True, seed=4)
    tables, pos, blk, blocks = place(starts, counts)
    args = (frequencies(128), tables.cuda(), i32(starts), cu_of(counts))
    pools = [[pool_for("bf16", blocks, 2, 128) for _ in (0, 1)] for _ in range(3)]
    out = nan_like(dq.contiguous())
    pk.rope_append_kv(*pools[0], out, dq, dk, dv, *args)
    pk.rope_append_kv(*pools[1], None, None, dk, dv, *args)
    pk.rope_append_kv(*pools[2], dq, dq, dk, dv, *args)          # queries turned where they are
    assert torch.equal(dq, out)
    for a in pools[1:]:
        assert torch.equal(a[0], pools[0][0]) and torch.equal(a[1], pools[0][1])


def test_rope_append_skips_rows_without_a_place():
    heads, counts = (4, 2, 64), [2, 2, 2, 2]
    (q, k, v), (dq, dk, dv) = rope_inputs("bf16", counts, heads, False, seed=6)
    tables = torch.tensor([[0, 1], [2, -1], [3, 4], [5, 6]], dtype=torch.int32).cuda()
    starts = [0, 15, 31, -1]          # the second's second row has no block, the third's no position
    kp, vp, out, err = pool_for("bf16", 7, 2, 64), pool_for("bf16", 7, 2, 64), nan_like(dq), err_flag()
    pk.rope_append_kv(kp, vp, out, dq, dk, dv, frequencies(64), tables, i32(starts), cu_of(counts), err_flag=err)
    assert int(err) == pk.DEV_ERR_BAD_BLOCK | pk.DEV_ERR_BAD_POS
    ok = [0, 1, 2, 4, 7]
    assert [bool(out[r].isnan().any()) for r in range(8)] == [r not in ok for r in range(8)]
    assert int((kp.abs().sum((1, 2, 4)) != 0).sum()) == len(ok)
    # rows behind the last sequence stay as they are, and the sum is flagged
    err.zero_()
    out = nan_like(dq)
    pk.rope_append_kv(kp, vp, out, dq, dk, dv, frequencies(64), tables[:2].contiguous(), i32([0, 0]), i32([0, 2, 3]), err_flag=err)
    assert int(err) == pk.DEV_ERR_BAD_CU
    assert [bool(out[r].isnan().any()) for r in range(8)] == [False] * 3 + [True] * 5


@pytest.mark.parametrize("cache", CACHES)
def test_rope_append_of_chunks_skips_what_has_no_place(cache):
    # chunks (block by block): a block without a table entry, positions before 0 and past the
    # table; every other row as if alone
    heads, counts, starts = (4, 2, 64), [20, 40, 30, 9], [0, 5, -7, 50]
    (q, k, v), (dq, dk, dv) = rope_inputs(cache, counts, heads, True, seed=8)
    tables = torch.arange(16, dtype=torch.int32).view(4, 4)
    tables[1, 1] = 16                                            # positions 16 .. 31 of sequence 1
    kp, vp, out, err = pool_for(cache, 16, 2, 64), pool_for(cache, 16, 2, 64), nan_like(dq.contiguous()), err_flag()
    args = (frequencies(64), tables.cuda(), i32(starts), cu_of(counts))
    rope_call(cache)(kp, vp, out, dq, dk, dv, *args, err_flag=err)
    assert int(err) == pk.DEV_ERR_BAD_BLOCK | pk.DEV_ERR_BAD_POS
    ok = [a + i >= 0 and a + i < 64 and not (s == 1 and 16 <= a + i < 32)
          for s, (a, n) in enumerate(zip(starts, counts)) for i in range(n)]
    assert [not bool(out[r].isnan().any()) for r in range(sum(counts))] == ok
    # one row per call and sequence gives the same pools and queries, bit for bit
    k2, v2, out2 = pool_for(cache, 16, 2, 64), pool_for(cache, 16, 2, 64), nan_like(out)
    for i in range(max(counts)):
        at = [(s, sum(counts[:s]) + i) for s in range(4) if i < counts[s]]
        rows = torch.tensor([r for _, r in at], device="cuda")
        one = torch.empty_like(out[rows])
        one.copy_(out2[rows])
        rope_call(cache)(k2, v2, one, dq[rows], dk[rows], dv[rows], frequencies(64),
                         tables[[s for s, _ in at]].contiguous().cuda(), i32([starts[s] + i for s, _ in at]), cu_of([1] * len(at)))
        out2[rows] = one
    assert torch.equal(kp, k2) and torch.equal(vp, v2)
    assert torch.equal(out.nan_to_num(7.0), out2.nan_to_num(7.0))
    # a prefix sum that does not end at the rows, or runs backwards
    for cu in ([0, 20, 60, 90, 98], [0, 20, 60, 90, 100], [0, 60, 20, 90, 99], [0, -4, 60, 90, 99]):
        err.zero_()
        out = nan_like(out)
        rope_call(cache)(kp, vp, out, dq, dk, dv, frequencies(64), tables.cuda(), i32([0, 5, 0, 40]), i32(cu), err_flag=err)
        assert int(err) & pk.DEV_ERR_BAD_CU


# ---------------------------------------------------------------------------- prefill
def run_prefill(c, starts, counts, q, window, sinks, scale, err=None, max_chunk=None, cu=None):
    out = nan_like(q.cuda())
    pk.prefill_attention_window(out, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(starts), cu_of(counts) if cu is None else cu,
                                scale, max_chunk or max(counts), window, sinks, err_flag=err)
    return out


def check_prefill(c, starts, counts, q, window, sinks, scale, out, every=1):
    row = 0
    for s, (a, n) in enumerate(zip(starts, counts)):
        pick = torch.arange(0, n, every)
        want, tol = attention(q[row:row + n][pick], c.k[s][:a + n], c.v[s][:a + n],
                              visible(a + pick, a + n, window, sinks), scale, "bf16", q.dtype)
        within(out[row:row + n].cpu()[pick], want, tol, f"sequence {s}")
        row += n


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads,rotary", [((4, 2, 64), 64), ((15, 3, 128), 112), ((2, 18, 64), 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_of_long_chunks_is_that_of_their_rows(cache, heads, rotary, interleaved):
    # 588 rows in one call go block by block, in calls of at most 230 row by row: the same queries,
    # pools and flags, also where a block has no table entry, before position 0 and past the table
    hq, hkv, d = heads
    counts, starts = [0, 230, 33, 1, 150, 64, 110], [5, 3, 0, 17, 70000, -9, 70199]
    (q, k, v), (dq, dk, dv) = rope_inputs(cache, counts, heads, True, seed=17)
    tables, _, _, blocks = place([max(0, x) for x in starts], counts)
    tables = tables[:, :4394].contiguous()                              # (70304 positions)
    tables[4, 70032 // BLOCK] = blocks
    freq, dt = frequencies(rotary), tables.cuda()
    got, flags = [], []
    for calls in ([range(7)], [[1], [2, 3], [0, 4], [5, 6]]):
        kp, vp = pool_for(cache, blocks, hkv, d), pool_for(cache, blocks, hkv, d)
        out, err = nan_like(dq.contiguous()), err_flag()
        for seqs in calls:
            seqs = list(seqs)
            a, b = sum(counts[:seqs[0]]), sum(counts[:seqs[-1] + 1])
            if seqs == [0, 4]:                                          # (all its rows are those of 4)
                a = sum(counts[:4])
            rope_call(cache)(kp, vp, out[a:b], dq[a:b], dk[a:b], dv[a:b], freq, dt[seqs], i32([starts[x] for x in seqs]),
                             cu_of([counts[x] for x in seqs]), interleaved, err_flag=err)
        got.append((kp, vp, out))
        flags.append(int(err))
    assert flags[0] == flags[1] == pk.DEV_ERR_BAD_BLOCK | pk.DEV_ERR_BAD_POS
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    ok = torch.tensor([0 <= a + i < 70304 and not (s == 4 and 70032 <= a + i < 70048)
                       for s, (a, n) in enumerate(zip(starts, counts)) for i in range(n)])
    out = got[0][2]
    assert torch.equal(out.isnan().any(-1).any(-1).cpu(), ~ok)
    at = torch.tensor([a + i for a, n in zip(starts, counts) for i in range(n)])
    want, size = rotated(q, at, freq.cpu(), interleaved)
    within(out[ok.cuda()], want[ok], (half_step(q.dtype) * want.abs() + 5e-7 * size + 1e-30)[ok], "queries")


@pytest.mark.parametrize("d", [64, 128])
def test_rope_append_fp8_codes_are_those_of_the_plain_append(d):
    # magnitudes over bf16's range, from row to row and within a row; infinities, NaN and zeros among the values
    g = torch.Generator().manual_seed(41)
    n, hkv = 1200, 2
    k, v = ((torch.randn(n, hkv, d, generator=g) * 2.0 ** torch.randint(-126, 120, (n, hkv, 1), generator=g)
             * 2.0 ** torch.randint(-12, 1, (n, hkv, d), generator=g)).bfloat16() for _ in range(2))
    v[5, 0], v[6, 1, 3], v[7, 0, 9], v[8, 1, 0] = 0.0, float("inf"), float("nan"), -float("inf")
    dk, dv = k.cuda(), v.cuda()
    for counts in ([1] * n, [n]):                                       # row by row, block by block
        blocks = sum((x + BLOCK - 1) // BLOCK for x in counts)
        tables = torch.arange(blocks, dtype=torch.int32).view(len(counts), -1).cuda()
        starts, cu = i32([0] * len(counts)), cu_of(counts)
        pools = [[pool_for("fp8", blocks, hkv, d) for _ in (0, 1)] for _ in (0, 1)]
        pk.rope_append_kv_fp8(*pools[0], None, None, dk, dv, frequencies(d), tables, starts, cu)
        pk.append_kv_fp8(*pools[1], dk, dv, tables, starts, cu)
        assert torch.equal(pools[0][1], pools[1][1])
        if len(counts) == n:
            # position 0 turns nothing: x1 1 - x2 0 is x1, but for an x1 of -0 (of the smallest
            # magnitudes here, rounded to bf16), which becomes +0 where x2 0 is -0
            for pool in (pools[0][0], pools[1][0]):
                codes = pool[..., :BLOCK * d]
                codes[codes == 0x80] = 0
            assert bool((k == 0).any()) and torch.equal(pools[0][0], pools[1][0])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (16, 0), (33, 4), (100, 17), (128, 70), (300, 0), (10**9, 0)])
def test_prefill_sees_the_window_and_the_sinks_only(heads, window, sinks):
    starts, counts = [0, 37, 200, 129, 5], [70, 1, 300, 0, 17]
    lens = [a + n for a, n in zip(starts, counts)]
    c = Cache("bf16", lens, heads, seed=window % 97 + sinks)
    q = c.queries(sum(counts))
    for s, (a, n) in enumerate(zip(starts, counts)):
        # a slot that no row of the chunk sees holds NaN, or its block is gone
        keep = visible(torch.arange(a, a + n), a + n, window, sinks).any(0) if n else torch.zeros(0, dtype=torch.bool)
        c.poison(s, keep)
    err = err_flag()
    out = run_prefill(c, starts, counts, q, window, sinks, 0.1, err)
    assert int(err) == 0
    check_prefill(c, starts, counts, q, window, sinks, 0.1, out)


def test_prefill_long_chunks_and_many_items():
    starts, counts = [1000, 0, 3], [900, 1500, 2100]
    c = Cache("bf16", [a + n for a, n in zip(starts, counts)], (8, 2, 128), seed=2)
    q = c.queries(sum(counts))
    for window, sinks, scale in ((512, 4, 0.1), (257, 0, -0.2), (1024, 130, 0.5)):
        out = run_prefill(c, starts, counts, q, window, sinks, scale)
        check_prefill(c, starts, counts, q, window, sinks, scale, out, every=7)
        for _ in range(3):
            assert torch.equal(run_prefill(c, starts, counts, q, window, sinks, scale), out)
    # more items than a schedule list holds: the strided walk
    counts = [3] * 260
    starts = [s % 50 for s in range(260)]
    c = Cache("bf16", [a + n for a, n in zip(starts, counts)], (12, 12, 64), seed=3, width=2000)
    q = c.queries(sum(counts))
    out = run_prefill(c, starts, counts, q, 20, 2, 0.1, max_chunk=400)
    check_prefill(c, starts, counts, q, 20, 2, 0.1, out)


def test_prefill_rows_agree_with_decode():
    starts, counts = [0, 300], [130, 40]
    c = Cache("bf16", [a + n for a, n in zip(starts, counts)], (14, 2, 64), seed=4)
    q = c.queries(sum(counts))
    out = run_prefill(c, starts, counts, q, 60, 5, 0.125)
    for row, s, p in ((0, 0, 0), (64, 0, 64), (129, 0, 129), (130, 1, 300), (169, 1, 339)):
        one = run_decode(c, [p + 1], q[row:row + 1], 60, 5, 0.125, tables=c.tables[s:s + 1])
        want, tol = attention(q[row:row + 1], c.k[s][:p + 1], c.v[s][:p + 1], visible(torch.tensor([p]), p + 1, 60, 5), 0.125,
                              "bf16", q.dtype)
        within(one, want, tol)
        within(out[row:row + 1], want, tol)


def test_prefill_leaves_the_rows_of_a_padded_batch():
    starts, counts = [10, 0], [40, 25]
    c = Cache("bf16", [50, 25], (8, 2, 128), seed=5)
    q = c.queries(65)
    good, err = run_prefill(c, starts, counts, q, 30, 4, 0.1), err_flag()
    padded = torch.full((100, 8, 128), float("nan")).to(torch.bfloat16)
    padded[:65] = q
    c.tables = torch.cat((c.tables, torch.full_like(c.tables, -1)))
    out = run_prefill(c, starts + [7, 9], counts, padded, 30, 4, 0.1, err, max_chunk=100, cu=i32([0, 40, 65, 65, 65]))
    assert int(err) == 0 and torch.equal(out[:65], good) and bool(out[65:].isnan().all())


def test_prefill_flags_bad_data():
    starts, counts = [10, 20, 30], [40, 40, 40]
    c = Cache("bf16", [50, 60, 70], (8, 2, 128), seed=6)
    q = c.queries(120)
    good, err = run_prefill(c, starts, counts, q, 30, 4, 0.1), err_flag()
    # a chunk that ends past q: flagged and left, the others computed
    out = run_prefill(c, starts, counts, q, 30, 4, 0.1, err, cu=i32([0, 40, 80, 121]), max_chunk=41)
    assert int(err) == pk.DEV_ERR_BAD_CU
    assert torch.equal(out[:80], good[:80]) and bool(out[80:].isnan().all())
    err.zero_()
    out = run_prefill(c, starts, counts, q, 30, 4, 0.1, err, max_chunk=33)
    assert int(err) == pk.DEV_ERR_HINT
    assert torch.equal(out[:33], good[:33]) and bool(out[33:40].isnan().all())
    err.zero_()
    out = run_prefill(c, [10, -1, 2**31 - 50], counts, q, 30, 4, 0.1, err)
    assert int(err) == pk.DEV_ERR_BAD_POS
    assert torch.equal(out[:40], good[:40]) and bool(out[40:].isnan().all())
    err.zero_()
    c.tables[1, 2] = -5
    out = run_prefill(c, starts, counts, q, 30, 4, 0.1, err)
    assert int(err) == pk.DEV_ERR_BAD_BLOCK and torch.equal(out[:40], good[:40])
    err.fill_(pk.DEV_ERR_TIMEOUT)
    assert bool(run_prefill(c, starts, counts, q, 30, 4, 0.1, err).isnan().all())


# ---------------------------------------------------------------------------- together
class Model:
    """One attention layer's path as a server runs it: rows enter rotated, in chunks and single
    tokens, and attend over the window; `rows` keeps what was entered, for the reference."""

    def __init__(self, cache, heads, window, sinks, seqs, tokens, seed):
        self.cache, self.window, self.sinks = cache, window, sinks
        self.hq, self.hkv, self.d = heads
        self.g = torch.Generator().manual_seed(seed)
        width = (tokens + BLOCK - 1) // BLOCK
        self.tables = torch.randperm(seqs * width, generator=self.g).int().view(seqs, width).cuda()
        self.kp, self.vp = (pool_for(cache, seqs * width, self.hkv, self.d) for _ in (0, 1))
        self.freq, self.scale = frequencies(self.d), self.d ** -0.5
        self.q, self.k, self.v = ([torch.zeros(0, h, self.d) for _ in range(seqs)] for h in (self.hq, self.hkv, self.hkv))
        self.wide = torch.float32 if cache == "f32" else torch.bfloat16
        self.err = err_flag()

    def step(self, counts):
        starts = [len(x) for x in self.k]
        n = sum(counts)
        x = torch.randn(n, self.hq + 2 * self.hkv, self.d, generator=self.g).to(self.wide)
        parts = torch.split(x.cuda(), (self.hq, self.hkv, self.hkv), 1)
        row = 0
        for s, m in enumerate(counts):
            for kept, part in zip((self.q, self.k, self.v), torch.split(x[row:row + m].float(), (self.hq, self.hkv, self.hkv), 1)):
                kept[s] = torch.cat((kept[s], part))
            row += m
        q, cu = torch.empty_like(parts[0].contiguous()), cu_of(counts)
        rope_call(self.cache)(self.kp, self.vp, q, *parts, self.freq, self.tables, i32(starts), cu, err_flag=self.err)
        out = nan_like(q)
        if all(m == 1 for m in counts):
            decode_call(self.cache)(out, q, self.kp, self.vp, self.tables, i32(a + 1 for a in starts), self.scale, self.window,
                                    self.sinks, err_flag=self.err)
        else:
            pk.prefill_attention_window(out, q, self.kp, self.vp, self.tables, i32(starts), cu, self.scale, max(counts),
                                        self.window, self.sinks, err_flag=self.err)
        return out

    def check(self, counts, out):
        """Against the definition on what was entered, in 64 bits.  Rotated rows stand in the
        cache and in q with one rounding each, so a score is off by at most 2 u sum |q k| scale
        (+ the next order), values by none: twice that per weight, on top of the usual."""
        row = 0
        for s, m in enumerate(counts):
            n = len(self.k[s])
            pos = torch.arange(n)
            k, _ = rotated(self.k[s], pos, self.freq.cpu(), False)
            q, _ = rotated(self.q[s][n - m:], pos[n - m:], self.freq.cpu(), False)
            u = half_step(self.wide)
            kk = k.abs().repeat_interleave(self.hq // self.hkv, 1)
            size = torch.einsum("rhd,nhd->rhn", q.abs(), kk).amax(-1) * self.scale
            want, tol = attention(q, k, self.v[s].double(), visible(pos[n - m:], n, self.window, self.sinks), self.scale,
                                  self.cache, self.wide)
            spread = self.v[s].abs().max()
            within(out[row:row + m], want, tol + (2 * 2.2 * u * size * spread)[..., None], f"sequence {s}")
            row += m


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_serving_run_in_chunks_and_tokens(cache):
    m = Model(cache, (8, 2, 128), 50, 4, 3, 400, seed=1)
    plan = [[1, 1, 1]] * 20 if cache == "f32" else [[100, 17, 64], [33, 1, 130]] + [[1, 1, 1]] * 20 + [[5, 1, 40], [1, 1, 1]]
    for counts in plan:
        out = m.step(counts)
        m.check(counts, out)
    assert int(m.err) == 0


@pytest.mark.parametrize("window,first", [(40, [70, 5, 33, 50]), (1100, [1300, 5, 900, 1500])])
def test_captured_step_follows_its_inputs(window, first):
    # one graph of append + attention, replayed as lengths grow; beside it the same on a
    # side stream without a graph
    m = Model("bf16", (8, 2, 128), window, 3, 4, max(first) + 40, seed=2)
    m.step(first)
    n, rows = 4, [torch.zeros(4, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)]
    starts, lens, cu = i32([0] * n), i32([0] * n), cu_of([1] * n)
    q, out = torch.empty_like(rows[0]), torch.empty_like(rows[0])
    kp2, vp2 = m.kp.clone(), m.vp.clone()

    def call(kp, vp, q, out):
        pk.rope_append_kv(kp, vp, q, *rows, m.freq, m.tables, starts, cu, err_flag=m.err)
        pk.decode_attention_window(out, q, kp, vp, m.tables, lens, m.scale, m.window, m.sinks, err_flag=m.err)

    at = [len(x) for x in m.k]
    starts.copy_(i32(at))
    lens.copy_(i32(a + 1 for a in at))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(m.kp, m.vp, q, out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(m.kp, m.vp, q, out)
    for _ in range(30):
        at = [len(x) for x in m.k]
        new = [torch.randn(n, h, 128, generator=m.g).to(torch.bfloat16) for h in (8, 2, 2)]
        for r, x in zip(rows, new):
            r.copy_(x)
        for s in range(n):
            for kept, x in zip((m.q, m.k, m.v), new):
                kept[s] = torch.cat((kept[s], x[s:s + 1].float()))
        starts.copy_(i32(at))
        lens.copy_(i32(a + 1 for a in at))
        graph.replay()
        got = out.clone()
        m.check([1] * n, got)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            q2, out2 = torch.empty_like(q), torch.empty_like(out)
            call(kp2, vp2, q2, out2)
        side.synchronize()
        assert torch.equal(out2, got)
    assert int(m.err) == 0


def test_bindings_take_the_same_calls_both_ways(monkeypatch):
    # the compiled way and the Python one: the same results, the same refusals
    from paged_kv_cache_207_gb300 import _native
    pk.lib()
    assert _native._quick is not None
    m = Model("bf16", (8, 2, 128), 40, 3, 2, 100, seed=5)
    q, k, v = (torch.randn(50, h, 128, generator=m.g).to(torch.bfloat16).cuda() for h in (8, 2, 2))
    starts, cu, lens, err = i32([0, 5]), cu_of([30, 20]), i32([30, 25]), err_flag()
    dq = torch.randn(2, 8, 128, generator=m.g).to(torch.bfloat16).cuda()

    def calls(**more):
        kp, vp, out, att, dec = m.kp.clone(), m.vp.clone(), nan_like(q), nan_like(q), nan_like(dq)
        pk.rope_append_kv(kp, vp, out, q, k, v, m.freq, m.tables, starts, cu, True, err, **more)
        pk.prefill_attention_window(att, out, kp, vp, m.tables, starts, cu, 0.1, 30, 2**40, 3, err, **more)
        pk.decode_attention_window(dec, dq, kp, vp, m.tables, lens, 1, 12, err_flag=err, **more)
        return kp, vp, out, att, dec

    quick = calls()
    for a, b in zip(quick, calls(stream=torch.cuda.current_stream())):     # an explicit stream: the Python way
        assert torch.equal(a, b)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = calls()
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(quick, got))
    fp8, f32 = pool_for("fp8", 4, 2, 128), pool_for("f32", 4, 2, 128)

    def refused():
        bad = [
            (TypeError, lambda: pk.decode_attention_window(dq.float(), dq, m.kp, m.vp, m.tables, lens, 0.1, 4)),
            (TypeError, lambda: pk.decode_attention_window(dq, dq, m.kp, m.vp, m.tables.long(), lens, 0.1, 4)),
            (ValueError, lambda: pk.decode_attention_window(dq, dq, m.kp, m.vp, m.tables, lens[:1], 0.1, 4)),
            (ValueError, lambda: pk.decode_attention_window(dq, dq, m.kp, m.vp[:3], m.tables, lens, 0.1, 4)),
            (ValueError, lambda: pk.decode_attention_window(dq.cpu(), dq, m.kp, m.vp, m.tables, lens, 0.1, 4)),
            (ValueError, lambda: pk.decode_attention_window(dq, q[::25], m.kp, m.vp, m.tables, lens, 0.1, 4)),
            (TypeError, lambda: pk.decode_attention_window(dq, dq, f32, f32, m.tables, lens, 0.1, 4)),
            (pk.PagedKVError, lambda: pk.decode_attention_window(dq, dq, m.kp, m.vp, m.tables, lens, 0.1, 0)),
            (pk.PagedKVError, lambda: pk.decode_attention_window(dq, dq, m.kp, m.vp, m.tables, lens, float("nan"), 4)),
            (ValueError, lambda: pk.decode_attention_window_fp8(dq, dq, m.kp, m.vp, m.tables, lens, 0.1, 4)),
            (ValueError, lambda: pk.rope_append_kv(m.kp, m.vp, None, q, k, v, m.freq, m.tables, starts, cu)),
            (TypeError, lambda: pk.rope_append_kv(m.kp, m.vp, q, q, k, v, m.freq.float(), m.tables, starts, cu)),
            (ValueError, lambda: pk.rope_append_kv(m.kp, m.vp, q, q, k, v[:49], m.freq, m.tables, starts, cu)),
            (ValueError, lambda: pk.rope_append_kv(m.kp, m.vp, q, q, k.transpose(1, 2).contiguous().transpose(1, 2), v, m.freq,
                                                   m.tables, starts, cu)),
            (pk.PagedKVError, lambda: pk.rope_append_kv(m.kp, m.vp, q, q, k, v, m.freq[:12], m.tables, starts, cu)),
            (TypeError, lambda: pk.rope_append_kv_fp8(fp8, fp8, q.float(), q, k, v, m.freq, m.tables, starts, cu)),
            (TypeError, lambda: pk.rope_append_kv(m.kp, m.vp, q, q, k, None, m.freq, m.tables, starts, cu)),
            (pk.PagedKVError, lambda: pk.prefill_attention_window(q.float(), q.float(), f32, f32, m.tables, starts, cu, 0.1, 30, 4)),
            (ValueError, lambda: pk.prefill_attention_window(q, q, m.kp, m.vp, m.tables, starts, cu[:2], 0.1, 30, 4)),
        ]
        for n, (kind, call) in enumerate(bad):
            with pytest.raises(kind):
                call()

    refused()
    monkeypatch.setattr(_native, "_quick", None)
    for a, b in zip(quick, calls()):
        assert torch.equal(a, b)
    refused()
    torch.cuda.synchronize()
    assert int(err) == 0


def test_offsets_past_32_bits():
    # pools of over 4 GiB each; the blocks in use are the last ones
    heads, blocks = (8, 8, 128), 140000
    kp, vp = (torch.empty(pk.pool_shape(blocks, 8, 128, torch.bfloat16), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    assert kp.numel() * 2 > 2**32
    n = 40
    tables = torch.tensor([[blocks - 1, blocks - 3, blocks - 2]], dtype=torch.int32)
    (q, k, v), (dq, dk, dv) = rope_inputs("bf16", [n], heads, False, seed=1)
    out, err = nan_like(dq), err_flag()
    pk.rope_append_kv(kp, vp, out, dq, dk, dv, frequencies(128), tables.cuda(), i32([0]), cu_of([n]), err_flag=err)
    small = [torch.stack([p[int(b)] for b in tables[0]]) for p in (kp, vp)]
    near = torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda()
    for window in (17, 100):
        got, want = torch.empty_like(dq), torch.empty_like(dq)
        pk.prefill_attention_window(got, out, kp, vp, tables.cuda(), i32([0]), cu_of([n]), 0.1, n, window, 2, err_flag=err)
        pk.prefill_attention_window(want, out, *small, near, i32([0]), cu_of([n]), 0.1, n, window, 2)
        assert torch.equal(got, want)
        pk.decode_attention_window(got[:1], out[:1].contiguous(), kp, vp, tables.cuda(), i32([n]), 0.1, window, 2, err_flag=err)
        pk.decode_attention_window(want[:1], out[:1].contiguous(), *small, near, i32([n]), 0.1, window, 2)
        assert torch.equal(got[0], want[0])
    want, size = rotated(k, torch.arange(n), frequencies(128).cpu(), False)
    stored = unpacked("bf16", small[0], 128, True).flatten(0, 1)[:n]
    within(stored, want, half_step(torch.bfloat16) * want.abs() + 5e-7 * size + 1e-30)
    assert int(err) == 0
