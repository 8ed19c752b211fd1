"""Measured cases of the sliding-window and rotary operators of the paged KV cache.

Three operators: appending keys and values with the position rotation applied on the way
(``rope_append_kv``, queries rotated in the same call), single-token attention over a
sliding window with a few first tokens that stay visible (``decode_attention_window``), and
the same mask for chunks of new tokens (``prefill_attention_window``).

``run`` computes them in plain torch operations, or, where ``own`` is true, through the
package.  Lengths come from the case alone (so ``work`` is exact), values and the placement
of blocks from the seed.  Only the blocks that an operator may read or write are in the
pools; table entries of positions that left the window are -1, as a cache that frees them
holds.
"""
import math
import random

import torch

own = False

BLOCK = 16
HEADS = ((32, 8, 128), (14, 2, 64), (12, 12, 64), (8, 1, 128), (16, 4, 128), (20, 4, 64), (9, 3, 128))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence: the latency of an interactive decode step
        _rope("rope one token", "bf16", 1, (14, 2, 64), 64, False, 1, 1, 700, 800, False, 1),
        # a serving batch's decode step: q, k and v are column ranges of one projection's
        # output, contexts up to 131072 tokens (far angles)
        _rope("rope batch step", "bf16", 256, (32, 8, 128), 128, False, 1, 1, 100, 131071, True, 2),
        # a step of chunked prefill
        _rope("rope chunks", "bf16", 16, (32, 8, 128), 128, False, 512, 512, 0, 3500, True, 3),
        # ragged chunks into an 8-bit cache, interleaved pairs over half the head
        _rope("rope ragged fp8", "fp8", 37, (32, 8, 128), 64, True, 1, 131, 0, 20000, False, 4),
        # one sequence, window filled: the smallest attention call of a decode step
        _decode("window one sequence", "bf16", 1, (14, 2, 64), 2500, 2600, 512, 4, 5),
        # a full serving batch of long contexts over a large window
        _decode("window batch", "bf16", 256, (32, 8, 128), 4500, 131071, 4096, 4, 6),
        # a mixed batch: empty, short and long contexts, an 8-bit cache
        _decode("window mixed fp8", "fp8", 64, (32, 8, 128), 0, 8000, 1024, 16, 7),
        # a 4-bit cache, odd window and sinks that end inside a block
        _decode("window fp4", "fp4", 128, (32, 8, 128), 1000, 16000, 2047, 5, 8),
        # full precision, one query head per kv head, no sinks
        _decode("window f32", "f32", 16, (12, 12, 64), 20, 1000, 256, 0, 9),
        # a few short ragged chunks, window smaller than some of them
        _prefill("window short chunks", 4, (14, 2, 64), 1, 70, 0, 500, 33, 4, 10),
        # a step of chunked prefill
        _prefill("window chunks", 16, (32, 8, 128), 512, 512, 0, 3584, 1024, 4, 11),
        # one long prompt in one call
        _prefill("window long prompt", 1, (32, 8, 128), 8192, 8192, 0, 0, 4096, 4, 12),
    ]


def _rope(name, cache, seqs, heads, rotary, interleaved, lo, hi, ctx_lo, ctx_hi, fused, mix):
    return {"name": name, "op": "rope", "cache": cache, "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "rotary": rotary, "interleaved": interleaved, "chunk_lo": lo, "chunk_hi": hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "fused": fused, "mix": mix}


def _decode(name, cache, seqs, heads, ctx_lo, ctx_hi, window, sinks, mix):
    return {"name": name, "op": "decode", "cache": cache, "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "window": window, "sinks": sinks, "mix": mix}


def _prefill(name, seqs, heads, lo, hi, ctx_lo, ctx_hi, window, sinks, mix):
    return {"name": name, "op": "prefill", "cache": "bf16", "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "chunk_lo": lo, "chunk_hi": hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "window": window, "sinks": sinks, "mix": mix}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "decode", "decode", "prefill"))
    heads = rng.choice(HEADS)
    mix = rng.randrange(1 << 20)
    if op == "rope":
        hi = rng.choice((1, _log(rng, 2, 700)))
        ctx = _log(rng, 16, 130000)
        rotary = rng.choice((heads[2], heads[2] // 2, heads[2] - 16))
        c = _rope("", rng.choice(("bf16", "bf16", "f32", "fp8")), _log(rng, 1, 256), heads, rotary, rng.random() < 0.4,
                  rng.randint(1, hi), hi, rng.randint(0, ctx), ctx, rng.random() < 0.5, mix)
    elif op == "decode":
        ctx = _log(rng, 1, 131071)
        c = _decode("", rng.choice(("bf16", "bf16", "fp8", "fp4", "f32")), _log(rng, 1, 256), heads, rng.randint(0, ctx), ctx,
                    _log(rng, 1, 4096), rng.choice((0, 1, 4, rng.randint(0, 70))), mix)
    else:
        hi = _log(rng, 1, 4000)
        ctx = _log(rng, 1, 8000)
        c = _prefill("", _log(rng, 1, 24), heads, rng.randint(1, hi), hi, rng.randint(0, ctx), ctx, _log(rng, 1, 4096),
                     rng.choice((0, 1, 4, rng.randint(0, 70))), mix)
    c.pop("name")
    most = max(_cost(x) for x in listed() if x["op"] == op)
    while _cost(c) > most and c["seqs"] > 1:
        c["seqs"] -= (c["seqs"] + 3) // 4
    while _cost(c) > most:
        for k in ("chunk_hi", "chunk_lo"):
            c[k] = max(1, c[k] // 2)
    return c


def _cost(c):
    """What the plain form moves (it works on padded sequences in 32 bits)."""
    starts, counts = _lengths(c)
    if c["op"] == "rope":
        return sum(counts) * (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"]
    if c["op"] == "decode":
        return c["seqs"] * _spread(c) * c["kv_heads"] * c["head_dim"]
    return c["seqs"] * max(counts) * _spread(c) * c["q_heads"]


def _lengths(c):
    """Per sequence: the tokens in the cache before the call, and the new ones (0 for decode,
    whose context counts its new token)."""
    r = random.Random(c["mix"])
    starts = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    if c["op"] == "decode":
        return starts, [0] * c["seqs"]
    counts = [r.randint(c["chunk_lo"], c["chunk_hi"]) for _ in range(c["seqs"])]
    return starts, counts


def _spread(c):
    """Positions per sequence that the plain form gathers: the sinks, then the window of the
    last token (decode) or of every row of the longest chunk."""
    starts, counts = _lengths(c)
    most = max(s + n for s, n in zip(starts, counts))
    reach = c["window"] if c["op"] == "decode" else c["window"] - 1 + max(counts)
    return min(c["sinks"], most) + min(reach, most)


def _live(c, s, start, count):
    """Blocks of a sequence that the call may read or write."""
    end = start + count
    if c["op"] == "rope":
        return list(range(start // BLOCK, (end + BLOCK - 1) // BLOCK))
    first = start - c["window"] if c["op"] == "decode" else start - c["window"] + 1
    sinks = range(0, (min(c["sinks"], end) + BLOCK - 1) // BLOCK)
    return sorted(set(sinks) | set(range(max(0, first) // BLOCK, (end + BLOCK - 1) // BLOCK)))


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    starts, counts = _lengths(c)
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    wide = torch.float32 if c["cache"] == "f32" else torch.bfloat16
    live = [_live(c, s, starts[s], counts[s]) for s in range(c["seqs"])]
    width = max(1, max(starts[s] + counts[s] + BLOCK - 1 for s in range(c["seqs"])) // BLOCK)
    blocks = max(1, sum(len(b) for b in live))
    place = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    at = torch.tensor([s * width + b for s in range(c["seqs"]) for b in live[s]], dtype=torch.int64, device=dev)
    tables = torch.full((c["seqs"] * width,), -1, dtype=torch.int32, device=dev)
    tables[at] = place[: at.numel()]
    state = {"case": c, "tables": tables.view(c["seqs"], width), "starts": torch.tensor(starts, dtype=torch.int32, device=dev),
             "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    if c["op"] != "rope":
        state["spread"] = _spread(c)
    if c["cache"] == "fp4":
        state["e2m1"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    total = sum(counts)
    state["cu"] = torch.tensor([sum(counts[:s]) for s in range(c["seqs"] + 1)], dtype=torch.int32, device=dev)
    state["k_pool"], state["v_pool"] = (_pool(c, blocks, g, i) for i in (0, 1))
    rows = c["seqs"] if c["op"] == "decode" else total
    if c["op"] == "rope":
        # float64 frequencies, base 500000: what a rotary model keeps
        state["inv_freq"] = torch.tensor([500000.0 ** (-2.0 * f / c["rotary"]) for f in range(c["rotary"] // 2)],
                                         dtype=torch.float64, device=dev)
        parts = (Hq, Hkv, Hkv)
        if c["fused"]:
            x = torch.randn((total, sum(parts), D), generator=g, device=dev, dtype=wide)
            state["q"], state["k_new"], state["v_new"] = torch.split(x, parts, dim=1)
        else:
            state["q"], state["k_new"], state["v_new"] = (
                torch.randn((total, h, D), generator=g, device=dev, dtype=wide) for h in parts)
        state["out"] = torch.empty((total, Hq, D), device=dev, dtype=wide)
    else:
        state["q"] = torch.randn((rows, Hq, D), generator=g, device=dev, dtype=wide)
        state["out"] = torch.empty_like(state["q"])
        state["scale"] = 1.0 / math.sqrt(D)
        state["max_chunk"] = max(counts)
    return state


def _pool(c, blocks, g, which):
    """A pool of N(0, 1) rows in the cache's type and layout (which: 0 keys, 1 values)."""
    Hkv, D = c["kv_heads"], c["head_dim"]
    dev = g.device
    if c["cache"] in ("bf16", "f32"):
        t = torch.bfloat16 if c["cache"] == "bf16" else torch.float32
        X = 8 if c["cache"] == "bf16" else 4
        return torch.randn((blocks, Hkv, D // X, BLOCK, X), generator=g, device=dev, dtype=t)
    x = torch.randn((blocks, Hkv, BLOCK, D), generator=g, device=dev)
    if c["cache"] == "fp8":
        scale = x.abs().amax(-1) / 448
        code = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        code = code.view(blocks, Hkv, BLOCK, D // 16, 16).transpose(2, 3) if which == 0 else code.transpose(2, 3)
        return torch.cat([code.reshape(blocks, Hkv, 16 * D), scale.view(torch.uint8).reshape(blocks, Hkv, 64)], -1).contiguous()
    # E2M1 codes with a power-of-two scale byte per 32 values of a row
    x = x.view(blocks, Hkv, BLOCK, D // 32, 32)
    byte = (torch.frexp(x.abs().amax(-1))[1] - 1 - 2 + 127).clamp(min=0)
    x = x * torch.exp2(127.0 - byte)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    code = (torch.bucketize(x.abs(), edges) + 8 * (x < 0)).to(torch.uint8).view(blocks, Hkv, BLOCK, D)
    if which == 0:    # [slot][c][ks][half] bytes of dims 16 ks + 8 half + 2 c, + 1
        pair = code.view(blocks, Hkv, BLOCK, D // 16, 2, 4, 2).permute(0, 1, 2, 5, 3, 4, 6)
    else:             # [r][c][mi][dh][half] bytes of slots 2 c + 8 half, + 1 of dim 16 mi + 8 dh + r
        pair = code.view(blocks, Hkv, 2, 4, 2, D // 16, 2, 8).permute(0, 1, 7, 3, 5, 6, 2, 4)
    packed = (pair[..., 0] | (pair[..., 1] << 4)).reshape(blocks, Hkv, 8 * D)
    return torch.cat([packed, byte.to(torch.uint8).reshape(blocks, Hkv, D // 2)], -1).contiguous()


# ---------------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "decode": _decode_plain, "prefill": _prefill_plain}[state["case"]["op"]](state)


def _run_own(s):
    import paged_kv_cache_207_gb300 as pk
    c = s["case"]
    quant = {"fp8": "_fp8", "fp4": "_fp4"}.get(c["cache"], "")
    if c["op"] == "rope":
        getattr(pk, "rope_append_kv" + quant)(
            s["k_pool"], s["v_pool"], s["out"], s["q"], s["k_new"], s["v_new"], s["inv_freq"], s["tables"], s["starts"],
            s["cu"], interleaved=c["interleaved"], err_flag=s["err"])
        return _rope_outputs(s, s["out"])
    if c["op"] == "decode":
        getattr(pk, "decode_attention_window" + quant)(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["starts"], s["scale"], c["window"], c["sinks"],
            err_flag=s["err"])
        return s["out"]
    pk.prefill_attention_window(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["starts"], s["cu"], s["scale"],
                                s["max_chunk"], c["window"], c["sinks"], err_flag=s["err"])
    return s["out"]


def _rope_outputs(s, q):
    c = s["case"]
    if c["cache"] != "fp8":
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    n = 16 * c["head_dim"]
    got = {"q": q}
    for name in ("k_pool", "v_pool"):
        got[name] = s[name][..., :n].view(torch.float8_e4m3fn)
        got[name + "_scales"] = s[name][..., n:].view(torch.float32)
    return got


def _rows(s, total):
    """Of each new row: its sequence, and its position."""
    row = torch.arange(total, device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    return seq, s["starts"].long()[seq] + row - s["cu"].long()[seq]


def _rope_plain(s):
    c = s["case"]
    R, D, Hkv = c["rotary"], c["head_dim"], c["kv_heads"]
    total = s["q"].shape[0]
    seq, pos = _rows(s, total)
    angle = pos.double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def rotated(x):
        x = x.float()
        y = x.clone()
        a, b = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        return y

    q = rotated(s["q"]).to(s["q"].dtype)
    k, v = rotated(s["k_new"]), s["v_new"].float()
    blk, slot = s["tables"][seq, pos // BLOCK].long(), pos % BLOCK
    if c["cache"] == "fp8":
        for pool, x, keys in ((s["k_pool"], k, True), (s["v_pool"], v, False)):
            scale = x.abs().amax(-1) / 448
            code = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
            codes = pool[..., : 16 * D]
            if keys:
                codes.unflatten(-1, (D // 16, BLOCK, 16))[blk, :, :, slot, :] = code.view(total, Hkv, D // 16, 16)
            else:
                codes.unflatten(-1, (D, BLOCK))[blk, :, :, slot] = code
            pool[..., 16 * D:].view(torch.float32)[blk, :, slot] = scale
    else:
        X = s["k_pool"].shape[-1]
        for pool, x in ((s["k_pool"], k), (s["v_pool"], v)):
            pool[blk, :, :, slot, :] = x.to(pool.dtype).view(total, Hkv, D // X, X)
    return _rope_outputs(s, q)


def _gather(s, pool, pos, seen, keys):
    """Rows [seqs][positions][Hkv][D] of a pool in 32 bits; zeros where not `seen`."""
    c = s["case"]
    D, Hkv = c["head_dim"], c["kv_heads"]
    seqs = torch.arange(c["seqs"], device=pos.device)[:, None]
    blk = torch.where(seen, s["tables"][seqs, pos // BLOCK].long(), 0)
    slot = torch.where(seen, pos % BLOCK, 0)
    if c["cache"] == "fp8":
        codes = pool[..., : 16 * D]
        if keys:
            code = codes.unflatten(-1, (D // 16, BLOCK, 16))[blk, :, :, slot, :].flatten(-2)
        else:
            code = codes.unflatten(-1, (D, BLOCK))[blk, :, :, slot]
        x = code.view(torch.float8_e4m3fn).float() * pool[..., 16 * D:].view(torch.float32)[blk, :, slot][..., None]
    elif c["cache"] == "fp4":
        n = 8 * D
        if keys:
            byte = pool[..., :n].unflatten(-1, (BLOCK, 4, D // 16, 2))[blk, :, slot].permute(0, 1, 2, 4, 5, 3)
            code = torch.stack((byte & 15, byte >> 4), -1).flatten(-4)
        else:
            view = pool[..., :n].unflatten(-1, (8, 4, D // 16, 2, 2))
            byte = view[blk, :, :, (slot % 8) // 2, :, :, slot // 8].permute(0, 1, 2, 4, 5, 3).flatten(-3)
            code = (byte >> (4 * (slot % 2))[..., None, None].to(torch.uint8)) & 15
        value = s["e2m1"][code.long()]
        scale = torch.exp2(pool[..., n:].unflatten(-1, (BLOCK, D // 32))[blk, :, slot].float() - 127)
        x = (value.unflatten(-1, (D // 32, 32)) * scale[..., None]).flatten(-2)
    else:
        x = pool[blk, :, :, slot, :].flatten(-2).float()
    return torch.where(seen[..., None, None], x.view(*pos.shape, Hkv, D), 0.0)


def _positions(s, first, end):
    """Positions the plain form looks at, [seqs][sinks + reach]: the sinks, then those from
    `first` on; and which of them lie in the cache, each once."""
    c = s["case"]
    dev = first.device
    spread = s["spread"]
    sinks = min(c["sinks"], spread)
    near = torch.clamp(first, min=0)[:, None] + torch.arange(spread - sinks, device=dev)
    far = torch.arange(sinks, device=dev).expand(c["seqs"], sinks)
    pos = torch.cat([far, near], 1)
    there = torch.cat([far < torch.minimum(torch.clamp(first, min=0), end)[:, None], near < end[:, None]], 1)
    return torch.where(there, pos, 0), there


def _softmax(x, seen):
    """Probabilities over the last axis of `x` where seen; zeros for a row that sees nothing."""
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def _decode_plain(s):
    c = s["case"]
    G = c["q_heads"] // c["kv_heads"]
    end = s["starts"].long()
    pos, seen = _positions(s, end - c["window"], end)
    k = _gather(s, s["k_pool"], pos, seen, True)
    v = _gather(s, s["v_pool"], pos, seen, False)
    q = s["q"].float().unflatten(1, (c["kv_heads"], G))
    x = torch.einsum("shgd,sthd->shgt", q, k) * s["scale"]
    p = _softmax(x, seen[:, None, None, :])
    return torch.einsum("shgt,sthd->shgd", p, v).flatten(1, 2).to(s["q"].dtype)


def _prefill_plain(s):
    c = s["case"]
    G = c["q_heads"] // c["kv_heads"]
    start, count = s["starts"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    pos, there = _positions(s, start - c["window"] + 1, start + count)
    k = _gather(s, s["k_pool"], pos, there, True)
    v = _gather(s, s["v_pool"], pos, there, False)
    seq, row_pos = _rows(s, s["q"].shape[0])
    i = row_pos - start[seq]
    q = s["q"].new_zeros((c["seqs"], s["max_chunk"]) + s["q"].shape[1:], dtype=torch.float32)
    q[seq, i] = s["q"].float()
    q = q.unflatten(2, (c["kv_heads"], G))
    at = start[:, None] + torch.arange(s["max_chunk"], device=pos.device)
    seen = pos[:, None, :] <= at[..., None]
    seen &= (pos[:, None, :] > at[..., None] - c["window"]) | (pos[:, None, :] < c["sinks"])
    seen &= there[:, None, :]
    x = torch.einsum("sihgd,sthd->shgit", q, k) * s["scale"]
    p = _softmax(x, seen[:, None, None])
    out = torch.einsum("shgit,sthd->sihgd", p, v).flatten(2, 3)
    return out[seq, i].to(s["q"].dtype)


# ---------------------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    starts, counts = _lengths(c)
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    e = 4 if c["cache"] == "f32" else 2
    # bytes of one token's keys or values of one head in the cache
    kept = {"f32": 4 * D, "bf16": 2 * D, "fp8": D + 4, "fp4": D // 2 + D // 32}[c["cache"]]
    if c["op"] == "rope":
        n = sum(counts)
        rows = n * (2 * Hq + 2 * Hkv) * D * e + n * 2 * Hkv * kept
        entries = sum(len(_live(c, s, starts[s], counts[s])) for s in range(c["seqs"]))
        return {"bytes": rows + 4 * entries + 8 * c["seqs"] + 4 * c["rotary"], "flops": 3 * n * (Hq + Hkv) * c["rotary"]}
    pairs = keys = entries = 0
    for s in range(c["seqs"]):
        a, b = starts[s], starts[s] + counts[s]
        entries += len(_live(c, s, a, counts[s]))
        if c["op"] == "decode":
            n = min(c["window"], b) + min(c["sinks"], max(0, b - c["window"]))
            pairs, keys = pairs + n, keys + n
        else:
            pairs += sum(min(c["window"], p + 1) + min(c["sinks"], max(0, p + 1 - c["window"])) for p in range(a, b))
            first = max(0, a - c["window"] + 1)
            keys += b - first + min(c["sinks"], first)
    rows = c["seqs"] if c["op"] == "decode" else sum(counts)
    return {"bytes": keys * 2 * Hkv * kept + 2 * rows * Hq * D * e + 4 * entries + 8 * c["seqs"], "flops": 4 * Hq * D * pairs}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_attention(case, s)


def _exact_rope(c, s):
    starts, counts = _lengths(c)
    R, D, X = c["rotary"], c["head_dim"], s["k_pool"].shape[-1]
    half = R // 2
    turn = torch.zeros((s["q"].shape[0], half), dtype=torch.complex128, device="cuda")
    blk, slot = [], []
    row = 0
    tables = s["tables"].cpu().tolist()
    for n, (a, m) in enumerate(zip(starts, counts)):
        p = torch.arange(a, a + m, dtype=torch.float64, device="cuda")
        t = p[:, None] * s["inv_freq"][None, :]
        turn[row:row + m] = torch.polar(torch.ones_like(t), t)
        blk += [tables[n][x // 16] for x in range(a, a + m)]
        slot += [x % 16 for x in range(a, a + m)]
        row += m
    blk, slot = torch.tensor(blk, device="cuda"), torch.tensor(slot, device="cuda")

    def spin(x):
        # the pair of each frequency as one complex number, turned
        x = x.double()
        pair = x[..., :R].reshape(*x.shape[:-1], half, 2) if c["interleaved"] else \
            torch.stack((x[..., :half], x[..., half:R]), -1)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None, :])
        y = y.flatten(-2) if c["interleaved"] else torch.cat((y[..., 0], y[..., 1]), -1)
        return torch.cat((y, x[..., R:]), -1)

    got = {"q": spin(s["q"])}
    for name, x in (("k_pool", spin(s["k_new"])), ("v_pool", s["v_new"].double())):
        if c["cache"] == "fp8":
            codes, scales = s[name][..., :16 * D].clone(), s[name][..., 16 * D:].clone().view(torch.float32).double()
            unit = x.abs().amax(-1) / 448
            value = (x / unit[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
            for d in range(D):
                place = (d // 16) * 256 + slot * 16 + d % 16 if name == "k_pool" else d * 16 + slot
                for h in range(c["kv_heads"]):
                    codes[blk, h, place] = value[:, h, d]
            for h in range(c["kv_heads"]):
                scales[blk, h, slot] = unit[:, h]
            got[name] = codes.view(torch.float8_e4m3fn).double()
            got[name + "_scales"] = scales
        else:
            pool = s[name].double()
            for d in range(D):
                pool[blk, :, d // X, slot, d % X] = x[:, :, d]
            got[name] = pool
    return got


def _unpacked(c, record, keys):
    """Blocks [n][Hkv][16][D] in 64 bits from their stored form."""
    D = c["head_dim"]
    n, H = record.shape[:2]
    out = torch.empty((n, H, 16, D), dtype=torch.float64, device=record.device)
    if c["cache"] in ("bf16", "f32"):
        X = record.shape[-1]
        for d in range(D):
            out[..., d] = record[:, :, d // X, :, d % X].double()
        return out
    t = torch.arange(16, device=record.device)
    if c["cache"] == "fp8":
        scale = record[..., 16 * D:].contiguous().view(torch.float32).double()
        for d in range(D):
            byte = record[..., (d // 16) * 256 + t * 16 + d % 16] if keys else record[..., d * 16 + t]
            out[..., d] = byte.contiguous().view(torch.float8_e4m3fn).double() * scale
        return out
    value = torch.tensor(E2M1, dtype=torch.float64, device=record.device)
    for d in range(D):
        if keys:
            byte = record[..., t * (D // 2) + ((d % 8) // 2) * (D // 8) + 2 * (d // 16) + (d % 16) // 8].long()
            code = byte >> 4 if d % 2 else byte & 15
        else:
            place = ((4 * (d % 8) + (t % 8) // 2) * (D // 16) + d // 16) * 4 + 2 * ((d % 16) // 8) + t // 8
            code = (record[..., place].long() >> (4 * (t % 2))) & 15
        scale = 2.0 ** (record[..., 8 * D + t * (D // 32) + d // 32].double() - 127)
        out[..., d] = torch.where(code >= 8, -1.0, 1.0) * value[code % 8] * scale
    return out


def _exact_attention(c, s):
    starts, counts = _lengths(c)
    G = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for n in range(c["seqs"]):
        a, m = starts[n], counts[n]
        if c["op"] == "decode":
            a, m = a - 1, 1      # the row is the context's last token
        if a >= 0:
            live = [b for b in _live(c, n, starts[n], counts[n])]
            where = s["tables"][n, torch.tensor(live, device="cuda")].long()
            k, v = (_unpacked(c, s[x][where], x == "k_pool").transpose(1, 2).flatten(0, 1) for x in ("k_pool", "v_pool"))
            j = (torch.tensor(live, device="cuda")[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
            p = torch.arange(a, a + m, device="cuda")[:, None]
            hidden = ~((j[None] <= p) & ((j[None] > p - c["window"]) | (j[None] < c["sinks"])))
            for h in range(c["kv_heads"]):
                for x in range(h * G, h * G + G):
                    w = torch.exp((s["q"][row:row + m, x].double() @ k[:, h].T * s["scale"]).masked_fill_(hidden, -1e300))
                    out[row:row + m, x] = (w @ v[:, h]) / w.sum(1, keepdim=True)
        row += m
    return out
