"""Calls around drafted trees that the bindings refuse, without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_207_gb300 import build, _native
    build.build()
    return _native


def test_compaction_into_a_table_without_columns(native):
    # its address is that of no table, which would mean in place
    i32 = torch.int32
    pool = torch.zeros(native.pool_shape(4, 2, 64, torch.bfloat16), dtype=torch.bfloat16)
    tables, start, cu, src = torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32), torch.arange(4, dtype=i32), torch.ones(3, dtype=i32)
    for call, pools in ((native.compact_kv, pool), (native.compact_kv_fp8, torch.zeros(native.fp8_pool_shape(4, 2, 64), dtype=torch.uint8)),
                        (native.compact_kv_fp4, torch.zeros(native.fp4_pool_shape(4, 2, 64), dtype=torch.uint8))):
        with pytest.raises(ValueError, match="dst_tables"):
            call(pools, pools, tables, src, start, cu, dst_tables=torch.zeros(3, 0, dtype=i32))


def test_truncate_takes_no_number_modulo_2_32(native):
    bm = native.BlockManager(8)
    a = bm.add_seq()
    bm.prepare_append(a, 0, 50)
    for seq, length in ((a, 2**32), (a, 2**32 + 5), (a, 5 - 2**32), (a, -2**32), (2**32 + a, 3), (a - 2**32, 3), (a, 2**70)):
        with pytest.raises(native.PagedKVError):
            bm.truncate(seq, length)
        assert bm.seq_len(a) == 50 and bm.stats()["free_blocks"] == 4
    bm.truncate(a, 50)
    bm.truncate(a, 17)
    assert bm.seq_len(a) == 17 and bm.stats()["free_blocks"] == 6


def test_tree_attention_refuses_tables_of_2_31_tokens(native):
    # the last tile of keys has to end within int32
    L = native.lib()

    def call(width):
        return L.pa_tree_attention(16, 16, 16, 16, 16, width, 16, 16, 16, 1, 1, 4, 0, 4, 2, 64, 8, 0.125, 1, 16, 1 << 30, None, None)

    assert [call(w) for w in (2**27 - 16, 2**27 - 15, 2**27 - 1, 2**27)] == [0, 1, 1, 1]
