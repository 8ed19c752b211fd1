"""A plain 64-bit implementation of the rotary append and of windowed attention, and small
inputs for them: contiguous logical rows, no paging, torch float64 on the CPU.

Tolerances are derived here once.  u(t) is half a step of type t relative to the value
(torch.finfo(t).eps / 2).

* Rotation: y = x1 cos - x2 sin.  cos and sin come within 1.3e-7 of the exact ones (the
  angle's last rounding 2.3e-8, the function 1 ulp, positions below 2^22), the two products
  and their sum add 2 u(f32) of |x1| + |x2|: 2.6e-7 (|x1| + |x2|), taken as 5e-7, then one
  rounding to the destination's type.
* Attention: out = sum w v / sum w.  A weight's relative error d gives at most 2 d A with
  A = sum w |v| / sum w.  d is the probability's rounding (bf16 for bf16 caches, f16 for the
  8- and 4-bit ones, fp32 for f32), plus twice the score's error (a dot of D products summed
  in fp32: D u(f32) times the largest sum of |q k| scale), plus 4e-6 for the exponential and
  the scale in log2 units.  The sums over n keys add n u(f32) A, the output one rounding.
  The 8- and 4-bit caches' probabilities also meet f16's smallest step: a probability times
  its value's scale and 2^8 is off by up to 2^-25 when it is below 2^-14.  Undoing the 2^8 and
  times the code that is 2^-33 448 per key for FP8; for FP4, whose largest scale is the one
  that becomes 2^8, it is 2^-33 6 times that scale, at most 2^-33 1.5 max |v| (a block's scale
  is at most a quarter of its largest value).  The sum of the weights is at least 1.
"""
from __future__ import annotations

import math

import torch

import paged_kv_cache_207_gb300 as pk

BLOCK = 16
U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rotated(x, positions, inv_freq, interleaved):
    """x [rows][heads][D] turned in 64 bits, and |x1| + |x2| of each element's plane."""
    x = x.double()
    R = 2 * inv_freq.shape[0]
    angle = positions.double()[:, None, None] * inv_freq.double()
    c, s = angle.cos(), angle.sin()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def visible(positions, length, window, sinks):
    """[rows][length]: which positions a row at each of `positions` sees."""
    j = torch.arange(length)
    p = positions[:, None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def attention(q, k, v, see, scale, cache, out_dtype):
    """q [rows][Hq][D], k, v [n][Hkv][D], see [rows][n]: outputs and their tolerance."""
    p_round = p_rounding(cache)
    rows, Hq, D = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    if n == 0:
        return out, tol + 1e-30
    for h in range(Hq):
        K, V, Q = k[:, h // G].double(), v[:, h // G].double(), q[:, h].double()
        K, V = torch.where(see.any(0)[:, None], K, 0.0), torch.where(see.any(0)[:, None], V, 0.0)
        x = torch.where(see, Q @ K.T * scale, -math.inf)
        top = x.amax(1, keepdim=True)
        w = torch.exp(x - torch.where(top.isinf(), 0.0, top))
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
        out[:, h] = w @ V
        A = w @ V.abs()
        size = torch.where(see, Q.abs() @ K.abs().T * abs(scale), 0.0).amax(1, keepdim=True)
        d = p_round + 2 * D * U32 * size + 4e-6
        tol[:, h] = half_step(out_dtype) * out[:, h].abs() + 2 * d * A * (1 + half_step(out_dtype)) + n * U32 * A + 1e-30
        tol[:, h] += n * 2.0 ** -33 * {"fp8": 448.0, "fp4": 1.5 * float(V.abs().max())}.get(cache, 0.0)
    return out, tol


def p_rounding(cache: str) -> float:
    return {"bf16": half_step(torch.bfloat16), "f32": 2 * U32}.get(cache, half_step(torch.float16))


def pool_for(cache, blocks, hkv, d, device="cuda"):
    if cache in ("bf16", "f32"):
        t = torch.bfloat16 if cache == "bf16" else torch.float32
        return torch.zeros(pk.pool_shape(blocks, hkv, d, t), dtype=t, device=device)
    shape = pk.fp8_pool_shape if cache == "fp8" else pk.fp4_pool_shape
    return torch.zeros(shape(blocks, hkv, d), dtype=torch.uint8, device=device)


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def unpacked(cache, pool, d, keys):
    """All rows of a pool as float64 [blocks][16][Hkv][D] on the CPU (and FP8 / FP4 scales)."""
    pool = pool.cpu()
    nb, hkv = pool.shape[:2]
    if cache in ("bf16", "f32"):
        return pool.double().permute(0, 3, 1, 2, 4).reshape(nb, BLOCK, hkv, d)
    if cache == "fp8":
        code = e4m3(pool[..., :16 * d].contiguous())
        code = (code.view(nb, hkv, d // 16, BLOCK, 16).permute(0, 3, 1, 2, 4) if keys else
                code.view(nb, hkv, d, BLOCK).permute(0, 3, 1, 2)).reshape(nb, BLOCK, hkv, d)
        scale = pool[..., 16 * d:].contiguous().view(torch.float32).double().permute(0, 2, 1)
        return code * scale[..., None]
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    out = torch.empty(nb, BLOCK, hkv, d, dtype=torch.float64)
    for t in range(BLOCK):
        for i in range(d):
            if keys:
                byte = pool[..., t * (d // 2) + ((i % 8) // 2) * (d // 8) + 2 * (i // 16) + (i % 16) // 8]
                code = byte >> 4 if i % 2 else byte & 15
            else:
                at = ((4 * (i % 8) + (t % 8) // 2) * (d // 16) + i // 16) * 4 + 2 * ((i % 16) // 8) + t // 8
                code = (pool[..., at] >> (4 * (t % 2))) & 15
            scale = 2.0 ** (pool[..., 8 * d + t * (d // 32) + i // 32].double() - 127)
            out[:, t, :, i] = value[code.long()] * scale
    return out


class Cache:
    """A paged cache of the given type with N(0, 1) rows: pools filled through the library's
    plain appends, `k` / `v` [seq] the stored values of every position in 64 bits."""

    def __init__(self, cache, lens, heads, seed=0, width=None, spare=3):
        self.cache, self.lens = cache, list(lens)
        self.hq, self.hkv, self.d = heads
        g = torch.Generator().manual_seed(seed)
        self.wide = torch.float32 if cache == "f32" else torch.bfloat16
        need = [(n + BLOCK - 1) // BLOCK for n in self.lens]
        self.width = width or max(1, max(need))
        self.blocks = sum(need) + spare
        perm = torch.randperm(self.blocks, generator=g).tolist()
        self.tables = torch.full((len(self.lens), self.width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for b in range(n):
                self.tables[s, b] = perm.pop()
        self.kp, self.vp = (pool_for(cache, self.blocks, self.hkv, self.d) for _ in (0, 1))
        total = sum(self.lens)
        rows = [torch.randn(total, self.hkv, self.d, generator=g).to(self.wide) for _ in (0, 1)]
        cu = [sum(self.lens[:i]) for i in range(len(self.lens) + 1)]
        self.cu = cu
        if total:
            append = {"fp8": pk.append_kv_fp8, "fp4": pk.append_kv_fp4}.get(cache, pk.append_kv)
            append(self.kp, self.vp, rows[0].cuda(), rows[1].cuda(), self.tables.cuda(),
                   torch.zeros(len(self.lens), dtype=torch.int32).cuda(), torch.tensor(cu, dtype=torch.int32).cuda())
        self.g = g
        self.refresh()

    def refresh(self):
        k, v = unpacked(self.cache, self.kp, self.d, True), unpacked(self.cache, self.vp, self.d, False)
        self.k, self.v = [], []
        for s, n in enumerate(self.lens):
            where = self.tables[s, : (n + BLOCK - 1) // BLOCK].long()
            self.k.append(k[where].flatten(0, 1)[:n])
            self.v.append(v[where].flatten(0, 1)[:n])

    def queries(self, rows):
        return torch.randn(rows, self.hq, self.d, generator=self.g).to(self.wide)

    def poison(self, s, keep):
        """Fill every slot of sequence s that `keep` ([positions], padded to its blocks) does not
        name with NaN (FP8: NaN codes and scales; FP4: its largest codes and scales), and drop
        the table entries of blocks without a kept slot."""
        n = self.tables.shape[1]
        for b in range(n):
            blk = int(self.tables[s, b])
            if blk < 0:
                continue
            slots = [t for t in range(BLOCK) if not (b * BLOCK + t < len(keep) and bool(keep[b * BLOCK + t]))]
            if len(slots) == BLOCK:
                self.tables[s, b] = -1
                continue
            for pool, keys in ((self.kp, True), (self.vp, False)):
                for t in slots:
                    self._poison_slot(pool[blk], t, keys)

    def _poison_slot(self, rec, t, keys):
        d = self.d
        if self.cache in ("bf16", "f32"):
            rec[:, :, t, :] = float("nan")
        elif self.cache == "fp8":
            if keys:
                rec[:, :16 * d].view(self.hkv, d // 16, BLOCK, 16)[:, :, t] = 0x7f
            else:
                rec[:, :16 * d].view(self.hkv, d, BLOCK)[:, :, t] = 0x7f
            rec[:, 16 * d + 4 * t: 16 * d + 4 * t + 4] = 0xff
        else:
            rec[:, 8 * d + t * (d // 32): 8 * d + (t + 1) * (d // 32)] = 0xff
            if keys:
                rec[:, t * (d // 2): (t + 1) * (d // 2)] = 0x77
            else:
                view = rec[:, :8 * d].view(self.hkv, 8, 4, d // 16, 2, 2)[:, :, (t % 8) // 2, :, :, t // 8]
                view |= 0x70 if t % 2 else 0x07


def decode_call(cache):
    return {"fp8": pk.decode_attention_window_fp8, "fp4": pk.decode_attention_window_fp4}.get(
        cache, pk.decode_attention_window)


def rope_call(cache):
    return {"fp8": pk.rope_append_kv_fp8, "fp4": pk.rope_append_kv_fp4}.get(cache, pk.rope_append_kv)


def within(got, want, tol, what=""):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside the tolerance, worst {float((off / tol).nan_to_num(1e9).max()):.3g} times")


def nan_like(t):
    """A buffer of NaN whose every element a kernel has to overwrite, or leave as it is."""
    return torch.full_like(t, float("nan"))
