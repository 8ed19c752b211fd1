"""The rotary append and the sliding-window attention where values leave the usual range, where
rows go by tiles, and where a sequence's parts do not divide evenly (tolerances: see
_window_common.py, and beside each test what it adds)."""
import math

import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _window_common import (BLOCK, Cache, attention, pool_for, visible, within)
from test_gpu_window import cu_of, frequencies, i32, run_decode

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
