// pa_rows.cuh -- where a new row goes: shared by the kernels that write rows into the pools.
#pragma once

#include "pa_internal.h"

namespace pa {

namespace {

__device__ __forceinline__ void raise_flag(int32_t* err, int bits) {
    if (err) atomicOr(err, bits);
}

// Sequence, position and physical block of new row `row` (reads only cu, start_pos
// and the tables, which no kernel of this library writes).  Flags and returns false
// when the row has no valid destination; `report` selects the thread that flags.  Params:
// tables, start_pos, cu, err, max_blocks, S (sequences), total (rows) and num_blocks.
template <typename Params>
__device__ __forceinline__ bool locate_row(const Params& p, int row, bool report, int& s_out,
                                           int& pos_out, int32_t& blk_out) {
    // sequence owning this row: cu[s] <= row < cu[s+1].  Guess by proportion (exact
    // when every sequence appends the same number of rows, e.g. one per decode step),
    // then fall back to a binary search.
    int s = (int)(((long long)row * p.S) / (p.total > 0 ? p.total : 1));
    if (s >= p.S) s = p.S - 1;
    int first = __ldg(p.cu + s);
    int next = __ldg(p.cu + s + 1);
    if (!(first <= row && row < next)) {
        int lo = 0, hi = p.S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.cu + mid) <= row) lo = mid;
            else hi = mid - 1;
        }
        s = lo;
        first = __ldg(p.cu + s);
        next = __ldg(p.cu + s + 1);
        if (row < first || row >= next) {
            if (report) raise_flag(p.err, PA_DEV_ERR_BAD_CU);
            return false;
        }
    }
    const long long pos = (long long)__ldg(p.start_pos + s) + (row - first);
    if (pos < 0 || pos >= (long long)p.max_blocks * kBlockTokens) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_POS);
        return false;
    }
    const int32_t blk = __ldg(p.tables + (size_t)s * p.max_blocks + (int)(pos / kBlockTokens));
    if (blk < 0 || blk >= p.num_blocks) {
        if (report) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
        return false;
    }
    s_out = s;
    pos_out = (int)pos;
    blk_out = blk;
    return true;
}

}  // namespace

}  // namespace pa
