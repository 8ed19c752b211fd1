"""Measured cases of what a paged KV cache does for drafted trees and for positions on several
axes.

Three operators: appending keys and values rotated by explicit positions on one or more axes
(``rope_append_kv_axes``, queries rotated in the same call), attention of a tree of new tokens
over the cache (``tree_attention``: every row sees what was there before and the tree's tokens
that its mask names), and moving rows of a sequence to consecutive positions (``compact_kv``,
in place or into other blocks).

``run`` computes them in plain torch operations, or, where ``own`` is true, through the
package.  Lengths, trees and the rows to move come from the case alone (so ``work`` is exact),
values and the placement of blocks from the seed.  Rows to move in place never lie where one is
moved to, except those that stay, so that a pass can be repeated.
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
        # one drafted tree of one sequence, rotated by depth: an interactive step
        _rope("axes one tree", "bf16", 1, (14, 2, 64), 64, False, 1, 16, 16, 700, 800, False, 1),
        # a serving batch's trees: q, k and v are column ranges of one projection's output,
        # contexts up to 131072 tokens (far angles)
        _rope("axes batch of trees", "bf16", 64, (32, 8, 128), 128, False, 1, 16, 32, 100, 131000, True, 2),
        # image prompts (time, height, width) into an 8-bit cache
        _rope("axes image prompts fp8", "fp8", 12, (32, 8, 128), 128, False, 3, 100, 1100, 0, 2000, False, 3),
        # one sequence, a small tree: the smallest attention call of a drafting step
        _tree("tree one sequence", "bf16", 1, (14, 2, 64), 500, 600, 8, 8, 4),
        # a serving batch, short to long contexts
        _tree("tree batch", "bf16", 64, (32, 8, 128), 500, 8000, 16, 32, 5),
        # wide trees: 256 query rows of a kv head
        _tree("tree wide", "bf16", 16, (32, 8, 128), 1000, 4000, 64, 64, 6),
        # few sequences with long contexts over an 8-bit cache
        _tree("tree long fp8", "fp8", 4, (32, 8, 128), 30000, 131000, 8, 16, 7),
        # a 4-bit cache
        _tree("tree fp4", "fp4", 32, (16, 4, 128), 1000, 16000, 24, 24, 8),
        # full precision, one query head per kv head, some trees of a single token
        _tree("tree f32", "f32", 8, (12, 12, 64), 20, 1000, 1, 21, 9),
        # the accepted paths of a serving batch move up behind their roots
        _compact("compact paths", "bf16", 64, (32, 8, 128), "path", 500, 8000, 1, 7, 10),
        # caches cut down to their first tokens and a window
        _compact("compact windows", "bf16", 16, (32, 8, 128), "window", 8300, 20000, 4096, 4100, 11),
        # a scattered half of ragged 8-bit caches, kept in blocks of its own
        _compact("compact scattered fp8", "fp8", 24, (16, 4, 128), "gather", 0, 9000, 0, 4000, 12),
    ]


def _rope(name, cache, seqs, heads, rotary, interleaved, axes, lo, hi, ctx_lo, ctx_hi, fused, mix):
    return {"name": name, "op": "rope", "cache": cache, "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "rotary": rotary, "interleaved": interleaved, "axes": axes, "rows_lo": lo, "rows_hi": hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "fused": fused, "mix": mix}


def _tree(name, cache, seqs, heads, ctx_lo, ctx_hi, lo, hi, mix):
    return {"name": name, "op": "tree", "cache": cache, "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "rows_lo": lo, "rows_hi": hi, "mix": mix}


def _compact(name, cache, seqs, heads, kind, ctx_lo, ctx_hi, lo, hi, mix):
    return {"name": name, "op": "compact", "cache": cache, "seqs": seqs, "q_heads": heads[0], "kv_heads": heads[1],
            "head_dim": heads[2], "kind": kind, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "rows_lo": lo, "rows_hi": hi, "mix": mix}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "tree", "tree", "tree", "compact"))
    heads = rng.choice(HEADS)
    mix = rng.randrange(1 << 20)
    if op == "rope":
        axes = rng.choice((1, 1, 2, 3))
        hi = _log(rng, 1, 1200 if axes > 1 else 64)
        ctx = _log(rng, 16, 130000)
        c = _rope("", rng.choice(("bf16", "bf16", "f32", "fp8")), _log(rng, 1, 128), heads,
                  rng.choice((heads[2], heads[2] // 2, heads[2] - 16)), rng.random() < 0.4, axes, rng.randint(1, hi), hi,
                  rng.randint(0, ctx), ctx, rng.random() < 0.5, mix)
    elif op == "tree":
        ctx, hi = _log(rng, 1, 131000), _log(rng, 1, 100)
        c = _tree("", rng.choice(("bf16", "bf16", "fp8", "fp4", "f32")), _log(rng, 1, 64), heads, rng.randint(0, ctx), ctx,
                  rng.randint(1, hi), hi, mix)
    else:
        kind = rng.choice(("path", "window", "gather"))
        if kind == "path":
            hi, ctx = _log(rng, 1, 32), _log(rng, 1, 20000)
        else:
            hi = _log(rng, 1, 5000)
            ctx = 2 * hi + _log(rng, 10, 12000)
        c = _compact("", rng.choice(("bf16", "bf16", "f32", "fp8")), _log(rng, 1, 64), heads, kind, rng.randint(0, ctx), ctx,
                     rng.randint(0, hi), hi, mix)
    c.pop("name")
    most = max(_cost(x) for x in listed() if x["op"] == op)
    while _cost(c) > most and c["seqs"] > 1:
        c["seqs"] -= (c["seqs"] + 3) // 4
    while _cost(c) > most:
        for k in ("ctx_hi", "ctx_lo", "rows_hi", "rows_lo"):
            c[k] = max(0 if k.endswith("lo") and op == "compact" else 1, c[k] // 2)
    return c


def _cost(c):
    """What the plain form moves (it works on padded sequences in 32 bits)."""
    starts, counts = _lengths(c)
    wide = c["seqs"] * c["kv_heads"] * c["head_dim"]
    if c["op"] == "rope":
        return sum(counts) * (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"]
    if c["op"] == "tree":
        most = max(a + n for a, n in zip(starts, counts))
        return most * (wide + c["seqs"] * max(counts) * c["q_heads"])
    return sum(a + n for a, n in zip(starts, counts)) * c["kv_heads"] * c["head_dim"] * (2 if c["cache"] == "f32" else 1)


def _lengths(c):
    """Per sequence: the tokens in the cache before the call, and the rows that it appends or
    attends from, or (compact) the rows it keeps."""
    r = random.Random(c["mix"])
    starts = [r.randint(c["ctx_lo"], max(c["ctx_lo"], c["ctx_hi"])) for _ in range(c["seqs"])]
    counts = [r.randint(c["rows_lo"], max(c["rows_lo"], c["rows_hi"])) for _ in range(c["seqs"])]
    return starts, counts


def _parents(c):
    """The drafted trees: the parent of each node (an earlier one), -1 for a root."""
    r = random.Random(c["mix"] + 1)
    return [[r.randint(max(-1, i - 8), i - 1) if i else -1 for i in range(n)] for n in _lengths(c)[1]]


def _moves(c):
    """Per sequence: the first position that rows move to, the positions they come from, and the
    sequence's tokens before the move."""
    r = random.Random(c["mix"] + 2)
    got = []
    for ctx, n in zip(*_lengths(c)):
        if c["kind"] == "path":        # the root stays, the others come from behind the path's end
            nodes = 3 * n + 4
            got.append((ctx, ([ctx] + sorted(r.sample(range(ctx + n, ctx + nodes), n - 1))) if n else [], ctx + nodes))
        elif c["kind"] == "window":    # the first four and the last ones
            sinks = min(4, ctx)
            n = max(0, min(n, (ctx - sinks) // 2))
            got.append((0, list(range(sinks)) + list(range(ctx - n, ctx)), ctx))
        else:                          # any of them, in order
            n = min(n, ctx)
            got.append((r.randint(0, 40), sorted(r.sample(range(ctx), n)), ctx))
    return got


def _ceil(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, D, S = c["q_heads"], c["kv_heads"], c["head_dim"], c["seqs"]
    wide = torch.float32 if c["cache"] == "f32" else torch.bfloat16
    starts, counts = _lengths(c)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    state = {"case": c, "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    moves = _moves(c) if c["op"] == "compact" else None
    if c["op"] == "compact":
        live = [range(_ceil(length)) for _, _, length in moves]
        counts = [len(src) for _, src, _ in moves]
    elif c["op"] == "rope":
        live = [range(a // BLOCK, _ceil(a + n)) for a, n in zip(starts, counts)]
    else:
        live = [range(_ceil(a + n)) for a, n in zip(starts, counts)]
    kept = [range(a // BLOCK, _ceil(a + len(src))) for a, src, _ in moves] if moves and c["kind"] == "gather" else []
    blocks = max(1, sum(map(len, live)) + sum(map(len, kept)))
    place = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)

    def table(lists, first):
        width = max([1] + [b[-1] + 1 for b in lists if len(b)])
        at = torch.tensor([s * width + b for s in range(S) for b in lists[s]], dtype=torch.int64, device=dev)
        t = torch.full((S * width,), -1, dtype=torch.int32, device=dev)
        t[at] = place[first:first + at.numel()]
        return t.view(S, width)

    state["tables"] = table(live, 0)
    state["cu"] = ints([sum(counts[:s]) for s in range(S + 1)])
    state["k_pool"], state["v_pool"] = (_pool(c, blocks, g, i) for i in (0, 1))
    total = sum(counts)
    if c["op"] == "compact":
        state["dst"] = table(kept, sum(map(len, live))) if kept else None
        state["starts"] = ints([a for a, _, _ in moves])
        state["src"] = ints([p for _, src, _ in moves for p in src])
        return state
    state["starts"] = ints(starts)
    if c["cache"] == "fp4":
        state["e2m1"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    if c["op"] == "tree":
        state["longest"] = max(a + n for a, n in zip(starts, counts))
        state["max_chunk"] = max(counts)
        words = (state["max_chunk"] + 31) // 32
        rows = []
        for tree in _parents(c):
            sees = []
            for i, up in enumerate(tree):
                sees.append((sees[up] if up >= 0 else 0) | 1 << i)
            rows += sees
        # (int32 words, as the machine holds them)
        state["mask"] = torch.tensor([[(m >> 32 * w & 0xffffffff) - (1 << 32 if m >> 32 * w + 31 & 1 else 0) for w in range(words)]
                                      for m in rows], dtype=torch.int64, device=dev).to(torch.int32).view(total, words)
        state["q"] = torch.randn((total, Hq, D), generator=g, device=dev, dtype=wide)
        state["out"] = torch.empty_like(state["q"])
        state["scale"] = 1.0 / math.sqrt(D)
        if own:
            import paged_kv_cache_207_gb300 as pk
            state["workspace"] = pk.tree_workspace(Hq, Hkv, D, state["max_chunk"])
        return state
    # float64 frequencies, base 500000: what a rotary model keeps
    R = c["rotary"]
    state["inv_freq"] = torch.tensor([500000.0 ** (-2.0 * f / R) for f in range(R // 2)], dtype=torch.float64, device=dev)
    state["positions"], state["plane_axis"] = ints(_positions(c)).view(c["axes"], total), ints(_plane_axis(c))
    parts = (Hq, Hkv, Hkv)
    if c["fused"]:
        x = torch.randn((total, sum(parts), D), generator=g, device=dev, dtype=wide)
        state["q"], state["k_new"], state["v_new"] = torch.split(x, parts, dim=1)
    else:
        state["q"], state["k_new"], state["v_new"] = (
            torch.randn((total, h, D), generator=g, device=dev, dtype=wide) for h in parts)
    state["out"] = torch.empty((total, Hq, D), device=dev, dtype=wide)
    return state


def _positions(c):
    """[axes][rows]: a tree's nodes at the context's length plus their depth, an image's at one
    time and a grid of 24 columns behind the text."""
    starts, counts = _lengths(c)
    if c["axes"] == 1:
        got = []
        for a, tree in zip(starts, _parents(c)):
            depth = []
            for up in tree:
                depth.append(depth[up] + 1 if up >= 0 else 0)
            got += [a + d for d in depth]
        return [got]
    grid = [(a, a + i // 24, a + i % 24) for a, n in zip(starts, counts) for i in range(n)]
    return [[x[k] for x in grid] for k in range(3)][:c["axes"]]


def _plane_axis(c):
    """The first quarter of the planes turns by the first axis, the rest by the others."""
    half = c["rotary"] // 2
    first = half // 4 if c["axes"] > 1 else half
    rest = half - first
    return [0] * first + [1 + f * (c["axes"] - 1) // rest for f in range(rest)]


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
    return {"rope": _rope_plain, "tree": _tree_plain, "compact": _compact_plain}[state["case"]["op"]](state)


def _run_own(s):
    import paged_kv_cache_207_gb300 as pk
    c = s["case"]
    quant = {"fp8": "_fp8", "fp4": "_fp4"}.get(c["cache"], "")
    if c["op"] == "rope":
        getattr(pk, "rope_append_kv_axes" + quant)(
            s["k_pool"], s["v_pool"], s["out"], s["q"], s["k_new"], s["v_new"], s["inv_freq"], s["plane_axis"],
            s["positions"], s["tables"], s["starts"], s["cu"], interleaved=c["interleaved"], err_flag=s["err"])
        return {"q": s["out"], **_pools(s)}
    if c["op"] == "tree":
        getattr(pk, "tree_attention" + quant)(
            s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["starts"], s["cu"], s["mask"], s["scale"],
            s["max_chunk"], s["workspace"], err_flag=s["err"])
        return s["out"]
    getattr(pk, "compact_kv" + quant)(
        s["k_pool"], s["v_pool"], s["tables"], s["src"], s["starts"], s["cu"], dst_tables=s["dst"], err_flag=s["err"])
    return _pools(s)


def _pools(s):
    c = s["case"]
    if c["cache"] != "fp8":
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    n = 16 * c["head_dim"]
    got = {}
    for name in ("k_pool", "v_pool"):
        got[name] = s[name][..., :n].view(torch.float8_e4m3fn)
        got[name + "_scales"] = s[name][..., n:].view(torch.float32)
    return got


def _rows(s, total):
    """Of each row: its sequence, and its place in the sequence's rows."""
    row = torch.arange(total, device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    return seq, row - s["cu"].long()[seq]


def _rope_plain(s):
    c = s["case"]
    R, D, Hkv = c["rotary"], c["head_dim"], c["kv_heads"]
    total = s["q"].shape[0]
    seq, i = _rows(s, total)
    pos = s["starts"].long()[seq] + i
    angle = s["positions"][s["plane_axis"].long()].double().T * s["inv_freq"]
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
    return {"q": q, **_pools(s)}


def _gather(s, pool, seq, pos, seen, keys):
    """Rows [positions][Hkv][D] of one sequence in 32 bits; zeros where not `seen`."""
    c = s["case"]
    D, Hkv = c["head_dim"], c["kv_heads"]
    blk = torch.where(seen, s["tables"][seq, pos // BLOCK].long(), 0)
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


def _tree_plain(s):
    c = s["case"]
    S, G, n = c["seqs"], c["q_heads"] // c["kv_heads"], s["max_chunk"]
    start, count = s["starts"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    dev = start.device
    pos = torch.arange(s["longest"], device=dev).expand(S, -1)
    there = pos < (start + count)[:, None]
    k, v = (_gather(s, s[x], torch.arange(S, device=dev)[:, None], pos, there, x == "k_pool") for x in ("k_pool", "v_pool"))
    seq, i = _rows(s, s["q"].shape[0])
    q = s["q"].new_zeros((S, n) + s["q"].shape[1:], dtype=torch.float32)
    q[seq, i] = s["q"].float()
    q = q.unflatten(2, (c["kv_heads"], G))
    mask = torch.zeros((S, n, s["mask"].shape[1]), dtype=torch.int32, device=dev)
    mask[seq, i] = s["mask"]
    # the tree's token at each position, and whether the row's bit for it is set
    j = (pos - start[:, None]).clamp(0, n - 1)
    word = torch.gather(mask, 2, (j // 32)[:, None, :].expand(S, n, -1))
    seen = (pos < start[:, None])[:, None, :] | ((word >> (j % 32)[:, None, :]) & 1).bool()
    seen &= there[:, None, :]
    x = torch.einsum("sihgd,sthd->shgit", q, k) * s["scale"]
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.einsum("shgit,sthd->sihgd", p, v).flatten(2, 3)
    return out[seq, i].to(s["q"].dtype)


def _compact_plain(s):
    c = s["case"]
    D = c["head_dim"]
    seq, i = _rows(s, s["src"].shape[0])
    a, b = s["src"].long(), s["starts"].long()[seq] + i
    from_blk, from_slot = s["tables"][seq, a // BLOCK].long(), a % BLOCK
    to_blk, to_slot = (s["tables"] if s["dst"] is None else s["dst"])[seq, b // BLOCK].long(), b % BLOCK
    if c["cache"] == "fp8":
        for pool, keys in ((s["k_pool"], True), (s["v_pool"], False)):
            codes, scales = pool[..., : 16 * D], pool[..., 16 * D:].unflatten(-1, (BLOCK, 4))
            if keys:
                codes = codes.unflatten(-1, (D // 16, BLOCK, 16))
                codes[to_blk, :, :, to_slot] = codes[from_blk, :, :, from_slot]
            else:
                codes = codes.unflatten(-1, (D, BLOCK))
                codes[to_blk, :, :, to_slot] = codes[from_blk, :, :, from_slot]
            scales[to_blk, :, to_slot] = scales[from_blk, :, from_slot]
    else:
        for pool in (s["k_pool"], s["v_pool"]):
            pool[to_blk, :, :, to_slot] = pool[from_blk, :, :, from_slot]
    return _pools(s)


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
        entries = sum(_ceil(a + m) - a // BLOCK for a, m in zip(starts, counts))
        return {"bytes": rows + 4 * entries + 8 * c["seqs"] + 6 * c["rotary"] + 4 * c["axes"] * n,
                "flops": 3 * n * (Hq + Hkv) * c["rotary"]}
    if c["op"] == "compact":
        moves = _moves(c)
        places = [(src[i], a + i) for a, src, _ in moves for i in range(len(src))]
        moved = sum(1 for a, b in places if a != b or c["kind"] == "gather")
        entries = sum(len({p // BLOCK for p in src}) + len({(a + i) // BLOCK for i in range(len(src))}) for a, src, _ in moves)
        return {"bytes": 2 * moved * 2 * Hkv * kept + 4 * len(places) + 4 * entries + 8 * c["seqs"], "flops": 0}
    keys = sum(a + n for a, n in zip(starts, counts))
    pairs = sum(a * n for a, n in zip(starts, counts))
    for tree in _parents(c):
        depth = []
        for up in tree:
            depth.append(1 + (depth[up] if up >= 0 else 0))
        pairs += sum(depth)
    rows, words = sum(counts), (max(counts) + 31) // 32
    entries = sum(_ceil(a + n) for a, n in zip(starts, counts))
    return {"bytes": keys * 2 * Hkv * kept + 2 * rows * Hq * D * e + 4 * entries + 4 * rows * words + 8 * c["seqs"],
            "flops": 4 * Hq * D * pairs}


# ---------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "compact": _exact_compact}[case["op"]](case, s)


def _exact_rope(c, s):
    starts, counts = _lengths(c)
    R, D, X = c["rotary"], c["head_dim"], s["k_pool"].shape[-1]
    half = R // 2
    turn = torch.empty((s["q"].shape[0], half), dtype=torch.complex128, device="cuda")
    where = _positions(c)
    for f, axis in enumerate(_plane_axis(c)):
        t = torch.tensor(where[axis], dtype=torch.float64, device="cuda") * s["inv_freq"][f]
        turn[:, f] = torch.polar(torch.ones_like(t), t)
    tables = s["tables"].cpu().tolist()
    places = [(tables[n][x // 16], x % 16) for n, (a, m) in enumerate(zip(starts, counts)) for x in range(a, a + m)]
    blk, slot = (torch.tensor([x[k] for x in places], device="cuda") for k in (0, 1))

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


def _exact_tree(c, s):
    starts, counts = _lengths(c)
    G = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for n, tree in enumerate(_parents(c)):
        a, m = starts[n], counts[n]
        where = s["tables"][n, :_ceil(a + m)].long()
        k, v = (_unpacked(c, s[x][where], x == "k_pool").transpose(1, 2).flatten(0, 1)[:a + m] for x in ("k_pool", "v_pool"))
        # each node sees the context, its ancestors and itself
        hidden = torch.ones((m, a + m), dtype=torch.bool)
        hidden[:, :a] = False
        for i in range(m):
            up = i
            while up >= 0:
                hidden[i, a + up] = False
                up = tree[up]
        hidden = hidden.cuda()
        for h in range(c["kv_heads"]):
            for x in range(h * G, h * G + G):
                w = torch.exp((s["q"][row:row + m, x].double() @ k[:, h].T * s["scale"]).masked_fill_(hidden, -1e300))
                out[row:row + m, x] = (w @ v[:, h]) / w.sum(1, keepdim=True)
        row += m
    return out


def _exact_compact(c, s):
    D = c["head_dim"]
    tables = s["tables"].cpu().tolist()
    dst = tables if s["dst"] is None else s["dst"].cpu().tolist()
    at = [(tables[n][p // 16], p % 16, dst[n][(a + i) // 16], (a + i) % 16)
          for n, (a, src, _) in enumerate(_moves(c)) for i, p in enumerate(src)]
    fb, fs, tb, ts = (torch.tensor([x[k] for x in at], dtype=torch.int64, device="cuda") for k in range(4))
    got = {}
    for name in ("k_pool", "v_pool"):
        if c["cache"] == "fp8":
            was = s[name][..., :16 * D].view(torch.float8_e4m3fn).double()
            now = was.clone()
            for d in range(D):
                x, y = ((d // 16) * 256 + fs * 16 + d % 16, (d // 16) * 256 + ts * 16 + d % 16) if name == "k_pool" else \
                    (d * 16 + fs, d * 16 + ts)
                now[tb, :, y] = was[fb, :, x]
            unit = s[name][..., 16 * D:].clone().view(torch.float32).double()
            moved = unit.clone()
            moved[tb, :, ts] = unit[fb, :, fs]
            got[name + "_scales"] = moved
        else:
            was = s[name].double()
            now = was.clone()
            for piece in range(was.shape[2]):
                now[tb, :, piece, ts] = was[fb, :, piece, fs]
        got[name] = now
    return got
