"""Tree attention whose waits run out: every call ends, says so in its flag, and leaves NaN or what a call that
goes well leaves, nothing else.

The kernels come from a build of their own in which a warp's waits for others give up after microseconds, so that
waits run out which would have ended.  No copy or product is lost: what is in flight is still waited for, as long
as ever, before a CTA ends."""
import ctypes
import os
import subprocess

import pytest
import torch

import paged_kv_cache_207_gb300 as pk
from paged_kv_cache_207_gb300 import build
from _tree_common import ancestors, packed, random_tree, rng_of
from _window_common import Cache, nan_like

pytestmark = pytest.mark.gpu

LIMITS = [100000, 20000, 10000, 5000, 3000, 2000, 1000, 500, 200, 0]      # ns
# pool type, heads, how far scales of values lie apart (in powers of two), nodes.  Sixteen nodes and more of four query heads
# have rows in all softmax warps, one node leaves most without; bf16 with more than 128 rows is the wide form.
KINDS = [("bf16", (8, 2, 128), 0, [1, 20, 0, 33, 2]), ("bf16", (8, 1, 64), 0, [60, 1, 17]), ("fp8", (8, 2, 128), 0, [1, 20, 0, 33, 2]),
         ("fp8", (4, 2, 64), 40, [3, 50, 1]), ("fp4", (8, 2, 128), 0, [1, 20, 0, 33, 2]), ("fp4", (4, 2, 64), 60, [3, 50, 1])]


@pytest.fixture(scope="module")
def tree(tmp_path_factory):
    at = str(tmp_path_factory.mktemp("waits") / "tree_waits.so")
    cmd = [build._nvcc(), "-shared", os.path.join(os.path.dirname(os.path.abspath(__file__)), "tree_waits.cu"), "-o", at, "-O3", "-std=c++17",
           "-Xcompiler", "-fPIC", "-I", build.INCLUDE, "-I", build.CSRC, "--expt-relaxed-constexpr"] + build.ARCH
    subprocess.run(cmd, check=True, capture_output=True)
    L, p, i32 = ctypes.CDLL(at), ctypes.c_void_p, ctypes.c_int32
    L.tree_waits_limit.argtypes = [ctypes.c_ulonglong]
    L.tree_waits_call.argtypes = [p] * 5 + [i32] + [p] * 3 + [i32] * 8 + [ctypes.c_float, i32] + [p] * 3
    return L


@pytest.mark.parametrize("cache,heads,spread,counts", KINDS)
def test_waits_that_run_out(tree, cache, heads, spread, counts):
    rng = rng_of("waits", cache, spread)
    counts = counts * 12
    ctx = [rng.choice([0, 40, 700, 2500]) for _ in counts]
    sees = [ancestors(random_tree(n, rng)) for n in counts]
    c = Cache(cache, [a + n for a, n in zip(ctx, counts)], heads, seed=80)
    if spread:
        k, v = (torch.randn(sum(c.lens), c.hkv, c.d, generator=c.g) for _ in (0, 1))
        v *= torch.exp2((torch.rand(len(v), generator=c.g) * spread).floor())[:, None, None]
        append = pk.append_kv_fp8 if cache == "fp8" else pk.append_kv_fp4
        append(c.kp, c.vp, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), c.tables.cuda(),
               torch.zeros(len(ctx), dtype=torch.int32, device="cuda"), torch.tensor(c.cu, dtype=torch.int32, device="cuda"))
    q = c.queries(sum(counts)).cuda()
    tables, start = c.tables.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
    cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    mask, ws = packed(sees).cuda(), pk.tree_workspace(*heads, max(counts))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dtype = {"bf16": 1, "fp8": 2, "fp4": 3}[cache]

    def run(limit, flag):
        out = nan_like(q)
        torch.cuda.synchronize()
        assert tree.tree_waits_limit(limit) == 0
        assert tree.tree_waits_call(out.data_ptr(), q.data_ptr(), c.kp.data_ptr(), c.vp.data_ptr(), tables.data_ptr(), tables.shape[1],
                                    start.data_ptr(), cu.data_ptr(), mask.data_ptr(), mask.shape[1], len(counts), sum(counts), max(counts),
                                    *heads, c.blocks, 0.1, dtype, ws.data_ptr(), None if flag is None else flag.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return out

    usual = 200000000
    good = run(usual, err)
    assert int(err) == 0 and bool(torch.isfinite(good).all())
    gave_up = 0
    for limit in LIMITS:
        for flag in (err, None, err):
            err.zero_()
            out = run(limit, flag)
            same = (out == good) | out.isnan()
            assert bool(same.all()), (limit, int((~same).sum()))
            if flag is not None:
                assert int(err) in (0, pk.DEV_ERR_TIMEOUT)
                assert int(err) or torch.equal(out, good)
                gave_up += int(err) != 0
    assert gave_up > 0
    err.zero_()
    assert torch.equal(run(usual, err), good) and int(err) == 0
