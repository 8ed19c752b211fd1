"""Tree attention over FP8 and MXFP4 pools whose rows' scales lie far apart: hidden nodes of any finite
size, and weight on rows that are small beside their neighbours.

Tolerances count what each row sees, and how much it weighs there.  With w the weights, A = sum w |v|
and B = sum w max_d |v| (what a token can add to any dim), u(t) half a step of type t:
* a weight's relative error d, twice over A: the probability's rounding u(f16), twice the score's error
  (D products summed in fp32, D u(f32) of the largest sum |q k| scale; FP8: 2^-17 of the row's largest query
  element times sum |k|; FP4: 2^-29 of it times D max |k|, and 2^-24 sum |q| max |k|, as a key's blocks are
  taken against its own largest one) and 4e-6 (exponential, scale in log2 units);
* n keys summed in fp32: n u(f32) A; the output's rounding;
* FP8: a value's scale rounded to f16 and its product with a code again, 2 u(f16) of A, and 2^-25 of the
  reference where that product is below f16's range.  A scale is 2^-14 of the reference at least and its
  row's largest value at least 2^8 of it: 2^-19 B.  FP4: blocks are taken exactly, or against their
  token's largest, off by 2^-25 of that one's scale times a code of up to 6, a quarter of which is less than
  max |v|: 2^-24 B;
* a probability times 2^7 is off by half of f16's smallest step, 2^-25: min(w, 2^-32) max_d |v| a key; where
  values' scales lie on the probabilities, the same of a unit of which the row's largest product of probability and
  scale is 2^-12 at least, times another key's code, at most 1.75 of that one's largest (448 over 256, 6 over 4): n 2^-19 B.
"""
import math

import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from _tree_common import U32, ancestors, packed, random_tree, rng_of, visible
from _window_common import Cache, half_step, nan_like, within

pytestmark = pytest.mark.gpu

CACHES = ["fp8", "fp4"]


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def cumulated(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def attention(q, k, v, see, scale, cache):
    """q [rows][Hq][D], k, v [n][Hkv][D], see [rows][n]: outputs and their tolerance."""
    rows, Hq, D = q.shape
    n, Hkv, _ = k.shape
    u16, ub = half_step(torch.float16), half_step(torch.bfloat16)
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for h in range(Hq):
        K, V, Q = (x.double() for x in (k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], q[:, h]))
        x = torch.where(see, Q @ K.T * scale, -math.inf)
        top = x.amax(1, keepdim=True)
        w = torch.exp(x - torch.where(top.isinf(), 0.0, top))
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
        out[:, h] = w @ V
        vmax = V.abs().amax(1)
        A, B = w @ V.abs(), (w @ vmax)[:, None]
        # (a weight of 0 needs no good score)
        near = see & (x > top - 120)
        size = torch.where(near, Q.abs() @ K.abs().T, 0.0).amax(1, keepdim=True) * abs(scale)
        kmax, k1 = (torch.where(near, y[None], 0.0).amax(1, keepdim=True) for y in (K.abs().amax(1), K.abs().sum(1)))
        qmax, q1 = Q.abs().amax(1, keepdim=True), Q.abs().sum(1, keepdim=True)
        score = D * U32 * size + abs(scale) * (qmax * k1 * 2.0 ** -17 if cache == "fp8" else
                                               D * qmax * kmax * 2.0 ** -29 + q1 * kmax * 2.0 ** -24)
        d = u16 + 2 * score + 4e-6
        tol[:, h] = ub * out[:, h].abs() + 2 * d * A * (1 + ub) + n * U32 * A + 1e-30
        tol[:, h] += 2 * u16 * A + 2.0 ** -19 * B if cache == "fp8" else 2.0 ** -24 * B
        tol[:, h] += (w.clamp(max=2.0 ** -32) @ vmax)[:, None] + n * 2.0 ** -19 * B
    return out, tol


def fill(c, k, v):
    """Rows [total][Hkv][D] of all sequences into the pools, by the plain append."""
    append = pk.append_kv_fp8 if c.cache == "fp8" else pk.append_kv_fp4
    append(c.kp, c.vp, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), c.tables.cuda(), i32([0] * len(c.lens)), i32(c.cu))
    c.refresh()


def run(c, ctx, sees, q, scale):
    counts = [x.shape[0] for x in sees]
    out, err = nan_like(q.cuda()), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = pk.tree_attention_fp8 if c.cache == "fp8" else pk.tree_attention_fp4
    call(out, q.cuda(), c.kp, c.vp, c.tables.cuda(), i32(ctx), i32(cumulated(counts)), packed(sees).cuda(), scale, max(counts),
         pk.tree_workspace(c.hq, c.hkv, c.d, max(counts)), err_flag=err)
    assert int(err) == 0
    return out


def rows_of(c, g):
    return [torch.randn(sum(c.lens), c.hkv, c.d, generator=g) for _ in (0, 1)]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("which", ["key", "value", "both"])
@pytest.mark.parametrize("exponent", [13, 30, 100, 120])
def test_a_hidden_node_of_any_size(cache, heads, which, exponent):
    # rows that do not see the node: it may be as large as the type allows
    ctx, counts, big = [70, 130, 0], [24, 40, 9], [(0, 5), (0, 23), (1, 0), (1, 39), (2, 8)]
    rng = rng_of("hidden", cache, heads)
    sees = [ancestors(random_tree(n, rng)) for n in counts]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=50)
    k, v = rows_of(c, c.g)
    for s, j in big:
        at = c.cu[s] + ctx[s] + j
        if which != "value":
            k[at] *= 2.0 ** exponent
        if which != "key":
            v[at] *= 2.0 ** exponent
    fill(c, k, v)
    q, cu, scale = c.queries(sum(counts)), cumulated(counts), heads[2] ** -0.5
    out = run(c, ctx, sees, q, scale)
    for s in range(len(ctx)):
        nodes = [j for x, j in big if x == s]
        clean = torch.nonzero(~sees[s][:, nodes].any(1)).flatten()
        assert 0 < len(clean) < counts[s]
        want, tol = attention(q[cu[s] + clean], c.k[s], c.v[s], visible(ctx[s], sees[s][clean]), scale, cache)
        within(out[cu[s] + clean.cuda()], want, tol, f"rows that do not see the nodes, sequence {s}")
        if which == "value":                 # and those that do see it have it
            seen = torch.nonzero(sees[s][:, nodes].any(1)).flatten()
            want, tol = attention(q[cu[s] + seen], c.k[s], c.v[s], visible(ctx[s], sees[s][seen]), scale, cache)
            within(out[cu[s] + seen.cuda()], want, tol, f"rows that see the nodes, sequence {s}")


# where the large values are among n tokens
LARGE = {
    "first": lambda n: torch.arange(n) < n // 2,
    "last": lambda n: torch.arange(n) >= n // 2,
    "tiles": lambda n: torch.arange(n) // 128 % 2 == 0,
    "tokens": lambda n: torch.arange(n) % 3 == 0,
    "one": lambda n: torch.arange(n) == n // 3,
}


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("exponent", [8, 20, 30, 70, 110])
@pytest.mark.parametrize("where", list(LARGE))
def test_weight_on_small_values(cache, exponent, where):
    # half of the rows look away from the tokens with large values (score -1000), half do not mind; many sequences,
    # so that a CTA has several tiles of one in turn
    heads, S = (4, 2, 64), 60
    rng = rng_of("small", cache, where)
    ctx, counts = [rng.randint(500, 900) for _ in range(S)], [rng.choice([1, 2, 3]) for _ in range(S)]
    sees = [ancestors(random_tree(n, rng)) for n in counts]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=51)
    k, v = rows_of(c, c.g)
    large = torch.cat([LARGE[where](n) for n in c.lens])
    v[large] *= 2.0 ** exponent
    k[:, :, 0] = torch.where(large, -200.0, 0.0)[:, None]
    fill(c, k, v)
    q, cu = c.queries(sum(counts)), cumulated(counts)
    q[:, :, 0] = 0.0
    q[:, 1::2, 0] = 40.0
    out = run(c, ctx, sees, q, 0.125)
    for s in range(S):
        rows = slice(cu[s], cu[s + 1])
        want, tol = attention(q[rows], c.k[s], c.v[s], visible(ctx[s], sees[s]), 0.125, cache)
        assert bool((want[:, 1::2].abs().amax() < 100) & (want[:, ::2].abs().amax() > 2.0 ** (exponent - 20)))
        within(out[rows], want, tol, f"sequence {s}")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("span", [60, 200])
@pytest.mark.parametrize("up", [True, False])
def test_sizes_that_drift(cache, up, span):
    # values grow or shrink by 2^span along the context and the weight is on either end of it
    heads, S, ctx = (4, 2, 128), 40, 1100
    c = Cache(cache, [ctx + 2] * S, heads, seed=52)
    k, v = rows_of(c, c.g)
    at = (torch.arange(ctx + 2) / ctx).repeat(S)
    v *= torch.exp2(span * (at if up else 1 - at) - span / 2)[:, None, None]
    k[:, :, 0] = (100 * at)[:, None]
    fill(c, k, v)
    q = c.queries(2 * S)
    q[:, 0::2, 0], q[:, 1::2, 0] = 30.0, -30.0
    sees = [ancestors([-1, 0])] * S
    out = run(c, [ctx] * S, sees, q, 0.1)
    for s in range(S):
        rows = slice(2 * s, 2 * s + 2)
        want, tol = attention(q[rows], c.k[s], c.v[s], visible(ctx, sees[s]), 0.1, cache)
        within(out[rows], want, tol, f"sequence {s}")


@pytest.mark.parametrize("cache", CACHES)
def test_rows_of_zeros(cache):
    # a scale of 0 is no small scale: single rows and whole tiles of zeros
    heads, S = (4, 2, 64), 60
    rng = rng_of("zeros", cache)
    ctx = [rng.randint(300, 900) for _ in range(S)]
    c = Cache(cache, [a + 3 for a in ctx], heads, seed=53)
    k, v = rows_of(c, c.g)
    for n, a in zip(c.lens, c.cu):
        none = (torch.arange(n) % 5 == 0) | (torch.arange(n) // 128 % 3 == 1)
        v[a:a + n][none] = 0.0
        k[a:a + n][torch.arange(n) % 7 == 0] = 0.0
    fill(c, k, v)
    q, sees = c.queries(3 * S), [ancestors([-1, 0, 0])] * S
    out = run(c, ctx, sees, q, 0.125)
    for s in range(S):
        rows = slice(3 * s, 3 * s + 3)
        want, tol = attention(q[rows], c.k[s], c.v[s], visible(ctx[s], sees[s]), 0.125, cache)
        within(out[rows], want, tol, f"sequence {s}")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("seed", range(6))
def test_sizes_at_random(cache, seed):
    # every token's key and value times a power of two of its own, from ranges that differ by sequence and by tile
    heads, S = [(4, 2, 64), (8, 1, 128), (3, 3, 64)][seed % 3], 50
    rng = rng_of("random", cache, seed)
    ctx, counts = [rng.choice([0, 30, 200, 500, 900]) for _ in range(S)], [rng.choice([1, 2, 7, 15]) for _ in range(S)]
    sees = [ancestors(random_tree(n, rng)) for n in counts]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=60 + seed)
    k, v = rows_of(c, c.g)
    for n, a in zip(c.lens, c.cu):
        for tile in range(0, n, 128):
            vs, ks, base = rng.choice([0, 0, 6, 16, 25, 60, 100]), rng.choice([0, 0, 3, 40, 90]), rng.choice([0, 0, 12, -30])
            rows = slice(a + tile, a + min(tile + 128, n))
            m = rows.stop - rows.start
            v[rows] *= torch.exp2((torch.rand(m, generator=c.g) * vs).floor() + base)[:, None, None]
            k[rows] *= torch.exp2(-(torch.rand(m, generator=c.g) * ks).floor())[:, None, None]
    fill(c, k, v)
    q, cu = c.queries(sum(counts)) * rng.choice([1, 4]), cumulated(counts)
    out = run(c, ctx, sees, q, 0.2)
    for s in range(S):
        rows = slice(cu[s], cu[s + 1])
        want, tol = attention(q[rows], c.k[s], c.v[s], visible(ctx[s], sees[s]), 0.2, cache)
        within(out[rows], want, tol, f"sequence {s}: {counts[s]} after {ctx[s]}")
