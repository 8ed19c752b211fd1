"""A plain 64-bit implementation of tree attention and of moving rows, with small trees.

Tolerances, derived here once; u(t) is half a step of type t relative to the value.

out = sum w v / sum w over the visible positions.  A weight's relative error d gives at most 2 d A
with A = sum w |v| / sum w.  d is the probability's rounding (bf16 for bf16 pools, f16 for the 8- and
4-bit ones, fp32 for f32) plus twice the score's error plus 4e-6 (exponential, scale in log2 units).
A score is a dot of D products summed in fp32: D u(f32) of size = max_t sum |q k| scale.  The sums
over n keys add n u(f32) A, the output one rounding.  Beyond that, where keys and values become f16
for the tensor cores:
* FP8: a value's code times its scale, the scale rounded to f16 and the product again: 2 u(f16) of A.
  Keys are taken as they are; a query element is two E4M3 numbers, the row's largest at 2^7 at least, exact
  but for what lies below E4M3's smallest step of 2^-9: 2^-17 of the largest.
* FP8 and FP4: a scale times the power of two that puts its tile's largest at 1 .. 2 (V: to 2^7, never
  below 1) is off by at most 2^-25 where it is below f16's normal range, and its code is at most 448,
  or 6, while max |k| is at least 448 or 4 of the largest scale's units: 1.5 2^-25 max |k|, with the product's
  own rounding taken as 2^-24 max |k| (and max |v|).
* a probability times 2^7 likewise, while the sum of the weights is at least 1: 2^-32 max |v| a key.
* a query element of FP4's, its row's largest at 2^4 at least: 2^-29 of the largest.
Pools whose largest magnitudes belong to rows outside the sequence are not used with these.
"""
from __future__ import annotations

import math
import random

import torch

from _window_common import BLOCK, U32, half_step, p_rounding


def random_tree(n, rng, spread=6):
    """Parents of n nodes: each an earlier one, or -1 for a root."""
    return [rng.randint(max(-1, i - spread), i - 1) if i else -1 for i in range(n)]


def ancestors(parents):
    """[n][n] bool: node i sees its ancestors and itself."""
    n = len(parents)
    see = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        up = i
        while up >= 0:
            see[i, up] = True
            up = parents[up]
    return see


def packed(sees, words=None):
    """int32 [rows][words] of the masks [n][n] of several sequences."""
    most = max([x.shape[1] for x in sees] + [1])
    words = words or (most + 31) // 32
    out = torch.zeros(sum(x.shape[0] for x in sees), words * 32, dtype=torch.int64)
    row = 0
    for x in sees:
        out[row:row + x.shape[0], : x.shape[1]] = x.long()
        row += x.shape[0]
    value = (out.view(-1, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(value >= 2**31, value - 2**32, value).to(torch.int32)


def visible(ctx, see):
    """[rows][ctx + n]: the context, then the nodes that the mask names."""
    return torch.cat([torch.ones(see.shape[0], ctx, dtype=torch.bool), see], 1)


def attention(q, k, v, see, scale, cache, out_dtype):
    """q [rows][Hq][D], k, v [n][Hkv][D], see [rows][n]: outputs and their tolerance."""
    rows, Hq, D = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    u16 = half_step(torch.float16)
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    quantised = cache in ("fp8", "fp4")
    for h in range(Hq):
        any_row = see.any(0)[:, None]
        K, V, Q = (x.double() for x in (k[:, h // G], v[:, h // G], q[:, h]))
        K, V = torch.where(any_row, K, 0.0), torch.where(any_row, V, 0.0)
        x = torch.where(see, Q @ K.T * scale, -math.inf)
        top = x.amax(1, keepdim=True)
        w = torch.exp(x - torch.where(top.isinf(), 0.0, top))
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
        out[:, h] = w @ V
        A = w @ V.abs()
        size = torch.where(see, Q.abs() @ K.abs().T * abs(scale), 0.0).amax(1, keepdim=True)
        score = D * U32 * size
        if cache == "fp8":
            k1 = torch.where(see, K.abs().sum(1)[None], 0.0).amax(1, keepdim=True)
            score = score + abs(scale) * Q.abs().amax(1, keepdim=True) * k1 * 2.0 ** -17
        if quantised:
            kmax, qmax = float(K.abs().max()), Q.abs().amax(1, keepdim=True)
            score = score + abs(scale) * (Q.abs().sum(1, keepdim=True) * kmax * 2.0 ** -24 + D * qmax * kmax * 2.0 ** -29)
        d = p_rounding(cache) + 2 * score + 4e-6
        tol[:, h] = half_step(out_dtype) * out[:, h].abs() + 2 * d * A * (1 + half_step(out_dtype)) + n * U32 * A + 1e-30
        if cache == "fp8":
            tol[:, h] += 2 * u16 * A
        if quantised:
            tol[:, h] += float(V.abs().max()) * (2.0 ** -24 + n * 2.0 ** -32)
    return out, tol


def moved(rows, tables, dst_tables, src, start):
    """Unpacked pool rows [blocks][16][..] after the moves (per sequence: source positions in order, first
    destination), every row read before any is written."""
    out = rows.clone()
    for s, (positions, a) in enumerate(zip(src, start)):
        for i, p in enumerate(positions):
            b = a + i
            out[int(dst_tables[s, b // BLOCK]), b % BLOCK] = rows[int(tables[s, p // BLOCK]), p % BLOCK]
    return out


def rng_of(*key):
    return random.Random("/".join(map(str, key)))
