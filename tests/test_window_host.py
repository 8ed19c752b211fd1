"""Refusals of the rotary append and of the windowed attention, without a GPU: host-checkable
faults return a status and launch nothing, and the bindings check tensors before any call."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_207_gb300 import build, _native
    build.build()
    return _native


def _rope(L, **kw):
    a = dict(kp=16, vp=16, qo=32, q=16, kn=16, vn=16, qos=256, qs=256, ks=128, vs=128, freq=16, R=64, il=0, tables=16, mb=4,
             start=16, cu=16, S=1, T=2, nb=8, Hq=4, Hkv=2, D=64, dtype=1)
    a.update(kw)
    return L.pa_rope_append_kv(*a.values(), None, None)


def test_rope_append_refusals(native):
    L = native.lib()
    assert _rope(L, S=0, T=0) == OK                            # nothing to do
    assert _rope(L, S=0) == INVALID
    for name in ("kp", "vp", "kn", "vn", "freq", "tables", "start", "cu"):
        assert _rope(L, **{name: None}) == INVALID, name
    for name in ("kp", "vp", "kn", "vn", "q", "qo"):
        assert _rope(L, **{name: 24}) == INVALID, name         # not on 16 bytes
    assert _rope(L, freq=12) == INVALID
    assert _rope(L, q=None) == INVALID and _rope(L, qo=None) == INVALID
    assert _rope(L, Hq=0) == INVALID and _rope(L, Hkv=0) == INVALID
    assert _rope(L, D=96) == UNSUPPORTED
    assert _rope(L, R=0) == INVALID and _rope(L, R=80) == INVALID and _rope(L, R=-16) == INVALID
    assert _rope(L, R=24) == UNSUPPORTED
    assert _rope(L, dtype=4) == INVALID and _rope(L, dtype=-1) == INVALID
    assert _rope(L, ks=127) == INVALID and _rope(L, vs=132) == INVALID     # overlapping, unaligned rows
    assert _rope(L, qs=200) == INVALID and _rope(L, qos=260) == INVALID
    assert _rope(L, dtype=0, qos=257) == INVALID
    assert _rope(L, qo=16, qos=512) == INVALID                 # in place with another stride
    assert _rope(L, mb=2**27) == INVALID and _rope(L, mb=0) == INVALID and _rope(L, nb=0) == INVALID
    assert _rope(L, T=-1) == INVALID and _rope(L, S=-1) == INVALID


def _decode(L, **kw):
    a = dict(out=16, q=16, k=16, v=16, tables=16, lens=16, S=1, Hq=4, Hkv=2, D=64, mb=4, nb=8, W=10, N=0, scale=0.125, dtype=1)
    a.update(kw)
    return L.pa_decode_attention_window(*a.values(), None, None)


def test_decode_window_refusals(native):
    L = native.lib()
    assert _decode(L, S=0) == OK
    for name in ("out", "q", "k", "v", "tables", "lens"):
        assert _decode(L, **{name: None}) == INVALID, name
    for name in ("out", "q", "k", "v"):
        assert _decode(L, **{name: 24}) == INVALID, name
    assert _decode(L, W=0) == INVALID and _decode(L, W=-3) == INVALID and _decode(L, N=-1) == INVALID
    assert _decode(L, D=32) == UNSUPPORTED and _decode(L, Hq=18) == UNSUPPORTED and _decode(L, Hq=5) == INVALID
    assert _decode(L, dtype=4) == INVALID
    assert _decode(L, scale=float("nan")) == INVALID and _decode(L, scale=float("inf")) == INVALID
    assert _decode(L, S=65536) == UNSUPPORTED and _decode(L, S=-1) == INVALID
    assert _decode(L, mb=2**27) == INVALID and _decode(L, nb=0) == INVALID


def _prefill(L, **kw):
    a = dict(out=16, q=16, k=16, v=16, tables=16, mb=4, start=16, cu=16, S=1, T=4, chunk=4, Hq=4, Hkv=2, D=64, nb=8, W=10, N=0,
             scale=0.125, dtype=1)
    a.update(kw)
    return L.pa_prefill_attention_window(*a.values(), None, None)


def test_prefill_window_refusals(native):
    L = native.lib()
    assert _prefill(L, S=0) == OK and _prefill(L, T=0) == OK and _prefill(L, chunk=0) == OK
    for name in ("out", "q", "k", "v", "tables", "start", "cu"):
        assert _prefill(L, **{name: None}) == INVALID, name
    for name in ("out", "q", "k", "v"):
        assert _prefill(L, **{name: 24}) == INVALID, name
    assert _prefill(L, W=0) == INVALID and _prefill(L, N=-1) == INVALID
    assert _prefill(L, dtype=0) == UNSUPPORTED and _prefill(L, dtype=2) == INVALID
    assert _prefill(L, D=96) == UNSUPPORTED and _prefill(L, Hq=18) == UNSUPPORTED and _prefill(L, Hq=5) == INVALID
    assert _prefill(L, scale=float("nan")) == INVALID and _prefill(L, mb=2**27) == INVALID


def test_bindings_check_the_tensors(native):
    bf16, i32 = torch.bfloat16, torch.int32
    pool = torch.zeros(native.pool_shape(4, 2, 64, bf16), dtype=bf16)
    q, new = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tables, lens, cu = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32), torch.arange(4, dtype=i32)
    freq = torch.ones(32, dtype=torch.float64)
    # tensors of the host are refused before any call
    with pytest.raises(ValueError):
        native.decode_attention_window(q.clone(), q, pool, pool, tables, lens, 0.1, 8)
    with pytest.raises(ValueError):
        native.prefill_attention_window(q.clone(), q, pool, pool, tables, lens, cu, 0.1, 1, 8)
    with pytest.raises(ValueError):
        native.rope_append_kv(pool, pool, q.clone(), q, new, new, freq, tables, lens, cu)
    with pytest.raises(ValueError):
        native.decode_attention_window(q.clone(), q[:2], pool, pool, tables, lens, 0.1, 8)
    with pytest.raises(ValueError):
        native.decode_attention_window(q.clone(), q, pool[0], pool[0], tables, lens, 0.1, 8)
    with pytest.raises(TypeError):
        native.decode_attention_window(q.clone(), q, pool.half(), pool.half(), tables, lens, 0.1, 8)
    with pytest.raises(ValueError):
        native.rope_append_kv(pool, pool, None, q, new, new, freq, tables, lens, cu)
    # types, shapes, layouts (checked before the device)
    dev = 0
    with pytest.raises(TypeError):
        native._checked(dev, lens.long(), "context_lens", i32, (3,))
    with pytest.raises(ValueError):
        native._checked(dev, lens, "context_lens", i32, (4,))
    with pytest.raises(TypeError):
        native._rows(dev, new.float(), "k_new", bf16, (3, 2, 64))
    with pytest.raises(ValueError):
        native._rows(dev, new, "k_new", bf16, (3, 2, 32))
    with pytest.raises(TypeError):
        native._rows(dev, None, "k_new", bf16, (3, 2, 64))
    assert native._bound(2**40) == 2**31 - 1 and native._bound(7) == 7


def test_visible_blocks_hold_every_visible_slot():
    """The list of blocks that the kernels walk, restated: every position that a row at first ..
    last sees is in it once, and it never passes the table."""
    block = 16
    for window in (1, 2, 15, 16, 17, 40, 10**6):
        for sinks in (0, 1, 15, 16, 17, 50, 10**6):
            for first in (0, 1, 16, 33, 100, 171):
                for last in (first, first + 1, first + 37):
                    low = max(0, first - window + 1)
                    n = min(sinks, low)
                    sink_blocks = n // block + (n % block != 0)
                    jump = max(0, low // block - sink_blocks)
                    count = last // block + 1 - jump
                    listed = [i if i < sink_blocks else i + jump for i in range(count)]
                    assert listed == sorted(set(listed)) and listed[-1] == last // block
                    seen = {j // block for p in range(first, last + 1) for j in range(p + 1) if j > p - window or j < sinks}
                    assert seen <= set(listed)
                    assert len(listed) <= len(seen) + 1
