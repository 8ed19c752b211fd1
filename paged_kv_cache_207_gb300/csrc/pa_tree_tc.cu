// pa_tree_tc.cu -- attention of a tree of drafted tokens over the paged cache on the 5th-generation
// tensor cores (bf16, FP8 and FP4 pools; the work's order: pa_tree.cuh).
//
// A CTA (one per SM) goes through its pieces: the rows of an item, one or two tiles of 128 (token,
// query head) rows of a kv head, against key tiles of 128 tokens (8 blocks),
//   S = Q K^T   into TMEM (one M128 N128 K16 MMA per 16 dims),
//   O += P V    into TMEM (one M128 N=D K16 MMA per block, P from TMEM over S's columns),
// with a running maximum per row that is raised only when a tile passes it by more than 2^8 (O is then
// rescaled).  A row belongs to two softmax threads (FP8: four) in warps of their own, each with a part of
// its columns.  Other warps make the bulk copies, issue all MMAs, copy K's pieces (bf16) or convert; a
// piece's first copies and scores run while the piece before it ends.  Keys before the tree take no mask;
// in the tree's own tiles a row's visible keys are its mask words, shifted to the tile, two instructions
// per score.
//
// Where it is bound.  bf16 to 128 rows: by the keys' bytes (64 sequences of 4096 tokens, 32 / 8 heads of
// 128: 1 node 166 us, 6.5 TB/s, 32 nodes 178).  bf16 with 256 rows: a key tile's MMAs take 1.5 us of the
// 2.0 that pass (64 nodes 227 us): scores of one row tile wait for its products with the values, as the TMEM
// holds one S tile per row tile.  FP8 (8 nodes 171, 32 nodes 181; four sequences of 80000: 188) and FP4 (184,
// 186; 196): 1.4 us a tile, which is how long the softmax, of which a tile is a chain (scores, maximum,
// agreement, exponentials, publication), takes beside the conversions on the same issue slots; without
// conversions 1.25, with the copies alone 1.05.
//
// bf16: K and V tiles come as they are (V's blocks by bulk copies; K's 16-byte pieces each to a
// place of their own, so that the tile is one operand of 128 rows).
//
// FP8: a record's keys are an E4M3 operand as they are stored, and a query row, eight significant bits,
// is the sum of two E4M3 numbers, exactly, but for elements below 2^-10 of the row's largest, which are off by 2^-17 of
// that at most: S takes two E4M3 MMAs for each one of 16-bit types, at twice the rate, nothing is converted, and a score
// is multiplied by its key's scale (against keys written as f16 operands: 187 us instead of 201 for four sequences of
// 30000 to 131000).  Probabilities do not fit E4M3 (flat rows of 10^5 keys lie below its range), so values are
// converted as FP4's are.
//
// FP4, and FP8's values: the records come by bulk copies and eight warps, one per block of the tile, write
// f16 operands (FP4: eight for K and eight for V).  f16 holds every code exactly.  An FP4 scale is a power
// of two and is folded in exactly; an FP8 scale is rounded to f16, and its product with a code again, each
// by 2^-11 of the value, an eighth of what bf16 probabilities would lose: to keep the scales of values
// apart would cost the softmax a product per probability.  An FP4 tile's K carries the power
// of two that puts its largest scale at 1 .. 2; the tile's scores take it back.  V's power of two is
// the piece's first tile's and changes, O with it, only where a tile's largest scale is 2^6 above or below.
// That holds for scales down to 2^-14 (FP4: 2^-23) of the reference, hidden tokens' included; a tile with others
// goes another way (wide_tile), with its columns' scales apart (against one reference alone, a hidden node of
// 2^30 the size of the rest made zeros of it, and values of 2^-20 of an earlier tile's lost most of their bits).
// Probabilities are taken times 2^7, at most 2^15, so that one below f16's normal range is off by at most 2^-32 of
// a weight of 1.  FP4's query rows become f16 times a power of two of their own, their largest element
// at 2^4 .. 2^5 (FP8: at 2^7 .. 2^8), and the row's scores give it back.
//
// Values of the tree's own tokens that are no finite numbers become zeros for the MMA (0 times an
// infinity would reach the rows that do not see the token); the rows that see them add them at the end.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "pa_tc.cuh"
#include "pa_tree.cuh"

namespace pa {

namespace {

// The longest wait of a warp for others, and of what is in flight before a CTA ends.
#ifdef PA_TREE_TEST_WAITS
__device__ uint64_t kWaitNs = 200000000ull;      // (a build of the tests' own, which set it)
#else
constexpr uint64_t kWaitNs = 200000000ull;
#endif
constexpr uint64_t kLandNs = 200000000ull;
constexpr int kTileRows = 128;
constexpr int kKeyBlocks = 8, kKeys = kKeyBlocks * kBlockTokens;
constexpr int kPieces = 4;                // records of pieces
constexpr float kRaise = 8.f;            // (log2) that a row's maximum lags at most

// Warps: the softmax, the copies (bf16: V's; else all records), the MMAs, then K's copies (bf16) or the
// conversions.  All have the registers of a launch of so many threads (128, 96 or 72: what setmaxnreg
// hands from role to role the compiler does not count on), so the softmax takes a row in pieces of 32
// columns: with two threads to a row from the TMEM once for the maximum and again for the
// probabilities, with four (FP8: 164 us instead of 183 for 64 sequences of 4096 tokens, 8 nodes) kept between.
// Four are too many warps beside FP4's conversions and two row tiles, and bf16 loses 1% to 2%.
template <pa_dtype T, int SW>
struct Roles {
    static constexpr int PARTS = T == PA_FP8_E4M3 ? 4 : 2;       // warps that share 32 rows
    static constexpr int SOFT = 4 * PARTS * SW, COPY = SOFT, MMA = SOFT + 1, FEED = SOFT + 2;
    static constexpr int FEEDS = T == PA_FP4_E2M1 ? 2 * kKeyBlocks : T == PA_FP8_E4M3 ? kKeyBlocks : SW == 1 ? 4 : 2;
    static constexpr int LEAD = FEED + FEEDS;          // (FP8, FP4) warps that the conversions wait for
    static constexpr int LEADS = T == PA_FP4_E2M1 ? 2 : T == PA_FP8_E4M3 ? 1 : 0;
    static constexpr int OTHERS = (2 + FEEDS + LEADS + 3) / 4 * 4;
    static constexpr int THREADS = (SOFT + OTHERS) * 32;
    static constexpr int READERS = SOFT + 1 + FEEDS + LEADS;       // of a piece's record: all but the copies' warp
};

template <int D, pa_dtype T, int SW>
struct Layout {
    static constexpr int TILE = kBlockTokens * D * 2;                  // a block's K or V as an operand
    static constexpr int KTILE = kKeyBlocks * TILE;
    static constexpr int QTILE = kTileRows * D * 2;                    // [D/8][16][8 rows][16 B]
    static constexpr bool RAW = T != PA_BF16;                          // values are converted
    static constexpr bool NAT = T == PA_FP8_E4M3;                      // keys are operands as they are
    static constexpr int REC = T == PA_BF16 ? TILE : T == PA_FP8_E4M3 ? 16 * D + 64 : 8 * D + D / 2;
    static constexpr int KST = RAW && !NAT ? 2 : 3, VST = RAW ? 2 : (SW == 1 || D == 64) ? 3 : 2;
    // stages of records (FP8: V's; FP4: K's and V's in turn): as many as find room, six at most
    static constexpr int HALF = kKeyBlocks * REC;
    static constexpr int KSTAGE = NAT ? HALF : KTILE;
    static constexpr int RST = !RAW ? 0 : NAT && D == 128 ? 4 : 6;
    // query rows: two row tiles: operands; one: on their way to the TMEM, [row][D / 8 pieces, turned by the row]
    static constexpr int Q = 0;
    static constexpr int K = Q + SW * QTILE;
    static constexpr int V = K + KST * KSTAGE;
    static constexpr int R = V + VST * KTILE;
    static constexpr int BAR = R + RST * HALF;
    static constexpr int NBAR = 52;
    // what the MMA warp passes on beside the results, and the search's scratch (once, before)
    static constexpr int SLOT = BAR + NBAR * 8;       // TMEM address
    static constexpr int ODD = SLOT + 16;             // [2] of a piece: values that are no finite numbers
    static constexpr int EXPS = ODD + 16;             // [8] (K, V) exponents of a tile, as the conversions leave them
    // as the MMA warp passes them on: FP4: [8]; FP8: [S tile][the columns' scales, the exponents]
    static constexpr int PASS = kKeys * 4 + 16;
    static constexpr int PASSED = EXPS + 64;
    static constexpr int SEEN = PASSED + (NAT ? 2 * PASS : 64);      // [8][8] a tile's block has such values
    static constexpr int TABLE = SEEN + 80;           // [8] FP4: a block's scales of values
    static constexpr int GONE = TABLE - 8;            // [2] the tile at which the conversions leave, K's and V's
    static constexpr int RECORDS = TABLE + (T == PA_FP4_E2M1 ? kKeyBlocks * 128 : 0);      // [kPieces] pieces
    static constexpr int FIRST = RECORDS + kPieces * 32;               // the CTA's first place, for a call that gives up
    static constexpr int ROWS = FIRST + 64;                            // [row tile][part][128] maxima, sums
    static constexpr int TOPS = ROWS + SW * Roles<T, SW>::PARTS * kTileRows * 4;     // [part][128] the queries' largest
    // wide tiles: FP8 [4] the columns' scales of values, FP4 [8] the columns' exponents, K's, then V's; [part][128] O's largest
    static constexpr int WIDE = TOPS + (RAW ? Roles<T, SW>::PARTS * kTileRows * 4 : 0);
    static constexpr int WIDE_TILES = NAT ? 4 : 8, WIDE_TILE = NAT ? kKeys * 4 : kKeys * 2;
    static constexpr int LARGEST = WIDE + (RAW ? WIDE_TILES * WIDE_TILE : 0);
    static constexpr int UNITS = LARGEST + (RAW ? Roles<T, SW>::PARTS * kTileRows * 4 : 0);      // of rows, where they differ
    static constexpr int BYTES0 = UNITS + (RAW ? Roles<T, SW>::PARTS * kTileRows * 4 : 0);
    static_assert(RECORDS % 16 == 0 && WIDE % 16 == 0);
    static_assert(BYTES0 <= 232448, "shared memory of one CTA");
    static_assert((Roles<T, SW>::THREADS / 32 + 6) * 8 <= KTILE, "the search's scratch, where the first tile goes");
    // one CTA (and its 512 TMEM columns) to an SM
    static constexpr int BYTES = BYTES0 < 122880 ? 122880 : BYTES0;
};

// barriers
constexpr int kKFull = 0, kKEmpty = 4, kVFull = 8, kVEmpty = 12, kRFull = 16, kREmpty = 22, kSFull = 28, kPFull = 30,
              kODone = 32, kPVDone = 34, kQFull = 35, kOFree = 37, kDone = 38, kEFull = 39,
              kXFull = 44, kXEmpty = 48;

// TMEM columns: two S tiles, O of each row tile; with one row tile, the query rows of two pieces.
constexpr uint32_t kColS = 0, kColO = 2 * kKeys, kColQ = kColO + 128;

constexpr uint32_t idesc(bool f16, int N, int b_mn_major) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(kTileRows >> 4) << 24);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint2 v) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// All lanes wait, a fifth of a second at most; the result is the same in all.  (A look costs four
// instructions: the waiting warps share their issue slots with those that work.)
//
// A warp that gives up raises the flag and waits for nothing any more, and what it does not do makes the others give up in
// their turn.  But a named barrier has no limit: who shares one with others comes to it as often as they do,
// whatever has become of its own waits (rows_leave, conversions_leave).
__device__ __noinline__ bool warp_wait_long(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    bool ok;
    do {
        int looks = 64;
        do ok = mbar_try_wait(bar, parity);
        while (!ok && --looks > 0);
    } while (!ok && global_timer_ns() - t0 < kWaitNs);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    // (a look gives each lane a result of its own: all have to go the same way)
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait_long(bar, parity);
}
// A named barrier of n threads that also says whether any of them brought `x`.
__device__ __forceinline__ bool named_bar_or(int id, int n, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "r"(n)
        : "memory");
    return r != 0u;
}
// One 32-byte store (the address a multiple of 32).
__device__ __forceinline__ void st_global_v8(void* addr, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// One lane of the warp, always the same one, in a form that the compiler sees to be one (MMAs issued
// under `lane == 0` take about 104 clocks each, and 150 in a loop, for the descriptors' way into uniform
// registers; under this and unrolled, 72 to 105, what the tensor cores take).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float pair_lo(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float pair_hi(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Bits of the halves of a 16-bit pair whose exponent is all ones.
__device__ __forceinline__ uint32_t not_finite(uint32_t x, uint32_t exponent) {
    const uint32_t e = x & exponent;
    return ((e & 0xffffu) == (exponent & 0xffffu) ? 0xffffu : 0u) | ((e >> 16) == (exponent >> 16) ? 0xffff0000u : 0u);
}

// Which of 32 keys from `node` on (below 0: of the context) a row sees of the tree's n nodes, whose mask is at `row`.
__device__ __forceinline__ uint32_t seen_word(const int32_t* row, int words, int node, int n) {
    const int left = n - node;
    uint32_t v = 0u;
    if (node < 0) {
        v = node <= -32 ? 0xffffffffu : ~(0xffffffffu << -node) | (uint32_t)__ldg(row) << -node;
    } else if (left > 0) {
        const uint32_t lo = (uint32_t)__ldg(row + node / 32);
        const uint32_t hi = (node & 31) != 0 && node / 32 + 1 < words ? (uint32_t)__ldg(row + node / 32 + 1) : 0u;
        v = __funnelshift_r(lo, hi, node & 31);
    }
    if (left < 32) v &= left > 0 ? ~(0xffffffffu << left) : 0u;
    return v;
}

// The conversions leave at tile t, for which a warp of theirs, or (done != 0) their lead, has given up.  gone: where
// the tile is said; go: their barriers, of tiles in turn; done: the barriers of their results, likewise.  A lead may be ahead:
// only when the conversions two tiles before are done is their barrier free, unless all leave there or before, and nobody
// waits at this one.
__device__ __noinline__ void conversions_leave(int t, uint32_t gone, uint32_t done, int go) {
    const uint64_t t0 = global_timer_ns();
    bool left = false;
    while (done != 0u && t >= 2) {
        int at;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(at) : "r"(gone) : "memory");
        left = __any_sync(0xffffffffu, at <= t - 2);
        if (left || __all_sync(0xffffffffu, mbar_test(done + 8 * (t & 1), ((t - 2) >> 1) & 1)) ||
            __any_sync(0xffffffffu, global_timer_ns() - t0 > kLandNs))
            break;
    }
    if (left) return;
    if ((threadIdx.x & 31) == 0) asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(gone), "r"(t) : "memory");
    __syncwarp();
    named_bar_arrive(go + (t & 1), 32 * (kKeyBlocks + 1));
}

// A run of key tiles of one item.
struct Piece {
    int j0, n;               // its first key tile, and how many; none: the CTA's work has ended
    int tokens, qrow;        // of the row tile, and the row of q of its first
    int start, nodes;        // of the sequence
    int s, h;                // sequence, kv head
    bool whole;              // all tiles of the item
    __device__ __forceinline__ int end() const { return start + nodes; }
    __device__ __forceinline__ int blocks() const { return (start + nodes + kBlockTokens - 1) / kBlockTokens; }
};
// The copies' warp goes through the places and leaves each piece as a record, one ahead of its own; the
// others read them (to find the next item costs a few hundred instructions and, at times, a load).
struct Walk {
    Cursor<kKeys> c;
    long long left;          // places from the cursor on
    __device__ __forceinline__ Piece piece(const TParams& p) const {
        Piece x;
        x.j0 = c.tile(c.at);
        const int j1 = c.tile((int)min((long long)c.cost(), c.at + left));
        x.n = left > 0 ? j1 - x.j0 : 0;
        x.tokens = item_tokens(p, c);
        x.qrow = c.q.q0 + c.rt * p.TQ;
        x.start = c.q.start;
        x.nodes = c.q.n;
        x.s = c.s;
        x.h = c.h;
        x.whole = x.j0 == 0 && j1 == c.q.tiles;
        return x;
    }
    // To the next item with tiles for this CTA (a run that ends before an item's first tile has none).
    __device__ __forceinline__ void next(const TParams& p) {
        left -= c.cost() - c.at;
        if (left > item_cost(kKeys)) next_item<kKeys>(p, c);
        else left = 0;
    }
};

static_assert(sizeof(Walk) <= 64, "its place in shared memory");

// The rest of a CTA's work for a softmax warp that has given up at tile `tile` of its piece ic (below 0: before the first
// queries): the barriers that it shares with the warps of its rows, in their order, then NaN for its rows.  first: where
// the CTA's work begins; row: the thread's, of the row tile; sum: its place for the row's sum; HALVES: row tiles.
template <int D, int HALVES, int PARTS, bool RAW>
__device__ __noinline__ void rows_leave(const TParams& p, const Walk* first, int ic, int tile, int row, int row_bar, float* sum) {
    const float nan = __int_as_float(0x7fc00000);
    const int lane = threadIdx.x & 31, tl = row / p.G, g = row - tl * p.G;
    auto busy = [&](const Piece& x) { return row - lane < x.tokens * p.G; };
    auto meet = [&](int times) {
        for (int k = 0; k < times; ++k) named_bar_sync(row_bar, 32 * PARTS);
    };
    // one row tile: queries through shared memory
    auto queries = [&](const Piece& x) {
        if (HALVES == 1 && x.n > 0 && busy(x)) meet(RAW ? 3 : 2);
    };
    Walk w = *first;
    for (int k = 0; k < ic; ++k) w.next(p);
    Piece x = w.piece(p);
    if (ic < 0) queries(x);
    for (; x.n > 0; tile = 0) {
        w.next(p);
        const Piece y = w.piece(p);
        const bool live = busy(x);
        for (int i = tile; i < x.n; ++i) {
            // two more where a row of theirs rises
            if (live && named_bar_or(row_bar, 32 * PARTS, false)) meet(2);
            if (i == 0) queries(y);
        }
        if (live) {
            *sum = nan;
            meet(1);
        }
        x = y;
    }
    // the rows of this piece and of the later ones are incomplete
    w = *first;
    for (int k = 0; w.left > 0; ++k, w.next(p)) {
        x = w.piece(p);
        if (k < ic || tl >= x.tokens) continue;
        if (!x.whole) {
            for (int i = 0; i < 2; ++i) p.part_ml[(size_t)(2 * blockIdx.x + i) * p.slot_rows + row] = make_float2(nan, nan);
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + ((size_t)(x.qrow + tl) * p.Hq + (size_t)x.h * p.G + g) * D);
        for (int v = 0; v < D / 8; ++v) dst[v] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    }
}

// The table of a piece in windows of 32 entries, one per lane, a window ahead of its use (read tile
// by tile, every tile would wait for a load).
struct Table {
    const int32_t* row;
    int first, nblk, lane, at;
    int32_t now, ahead;
    __device__ __forceinline__ int32_t fetch(int w) const {
        const int b = first + 32 * w + lane;
        return b < nblk ? __ldg(row + b) : -1;
    }
    __device__ __forceinline__ Table(const TParams& p, const Piece& x, int lane_) {
        row = p.tables + (size_t)x.s * p.max_blocks;
        first = x.j0 * kKeyBlocks;
        nblk = x.blocks();
        lane = lane_;
        at = 0;
        now = fetch(0);
        ahead = fetch(1);
    }
    // Entry of block `lane % 8` of the piece's i-th tile (in order); -1: past the last, or no block of
    // the pool (flagged).  The whole warp.
    __device__ __forceinline__ int32_t block(const TParams& p, int i) {
        while (i / 4 > at) {
            now = ahead;
            ++at;
            ahead = fetch(at + 1);
        }
        const int b = lane & (kKeyBlocks - 1);
        int32_t blk = __shfl_sync(0xffffffffu, now, (i % 4) * kKeyBlocks + b);
        if (first + i * kKeyBlocks + b >= nblk) return -1;
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane < kKeyBlocks) raise_flag(p.err, PA_DEV_ERR_BAD_BLOCK);
            blk = -1;
        }
        return blk;
    }
};

// What the conversions' lead and the MMA warp say of a tile beside its values' exponent of 8 bits: it is a wide one
// (wide_tile), with its values' own scales, its keys'; then V's reference is in bits 8 .. 15 of its keys' exponent.
constexpr uint32_t kWideValues = 1u << 8, kWideKeys = 1u << 9;

// The conversions of one block of a tile by one warp: K to [D/8][8 blocks][16 slots][8 dims], V to
// [16 token groups of 8][D/8][8 dims][8 tokens], f16.  `live`: its tokens that are keys; `own`: those of the tree.
template <int D, pa_dtype T>
struct Convert;

template <int D>
struct Convert<D, PA_FP8_E4M3> {
    static constexpr int DEPTH = 14;           // how far scales lie below the largest in a tile that is not wide
    // A lane's four scales of a tile, without their signs; 0 where they are no keys' or not finite.
    struct Scales { uint32_t x[4]; };
    static __device__ __forceinline__ Scales scales(uint32_t raw, int rec, int keys, int lane) {
        const uint4 y = ld_shared_v4(raw + (lane >> 2) * rec + 16 * D + (lane & 3) * 16);
        const int n = keys - 4 * lane;                                     // keys of this lane's four
        auto of = [&](uint32_t z, int i) { return n > i && (z & 0x7f800000u) != 0x7f800000u ? z & 0x7fffffffu : 0u; };
        return Scales{{of(y.x, 0), of(y.y, 1), of(y.z, 2), of(y.w, 3)}};
    }
    // Their largest biased exponent.
    static __device__ __forceinline__ int exponent(const Scales& s) {
        return (int)(__reduce_max_sync(0xffffffffu, max(max(s.x[0], s.x[1]), max(s.x[2], s.x[3]))) >> 23);
    }
    // Whether one of the lane's that is not 0 has an exponent below e.
    static __device__ __forceinline__ bool below(const Scales& s, int e) {
        const uint32_t least = e > 0 ? ((uint32_t)e << 23) - 1u : 0u;      // (less 1: a scale of 0 passes to the top)
        return min(min(s.x[0] - 1u, s.x[1] - 1u), min(s.x[2] - 1u, s.x[3] - 1u)) < least;
    }
    // A wide tile's scales of values as its columns lie (the keys' lie so too), 0 where the tree's own (from the ctx-th
    // on) are not finite; in the record 1 takes their place, so that the operands are the codes.
    static __device__ __forceinline__ void widen(uint32_t raw, int rec, uint32_t to, int keys, int ctx, int lane) {
        const uint32_t at = raw + (lane >> 2) * rec + 16 * D + (lane & 3) * 16;
        const uint4 y = ld_shared_v4(at);
        auto finite = [](uint32_t z) { return (z & 0x7f800000u) != 0x7f800000u; };
        auto keep = [&](uint32_t z, int i) { return 4 * lane + i < keys && (4 * lane + i < ctx || finite(z)) ? z : 0u; };
        auto one = [&](uint32_t z) { return finite(z) && (z << 1) != 0u ? 0x3f800000u : z; };
        st_shared_v4(to + ((lane >> 1) & 1) * 256 + (lane >> 2) * 32 + (lane & 1) * 16,
                     make_uint4(keep(y.x, 0), keep(y.y, 1), keep(y.z, 2), keep(y.w, 3)));
        st_shared_v4(at, make_uint4(one(y.x), one(y.y), one(y.z), one(y.w)));
    }
    static __device__ __forceinline__ bool values(uint32_t raw, uint32_t dst, uint32_t, int rv, int lane, uint32_t live, uint32_t own) {
        const float f = exp2i(127 - rv);
        uint4 code[D / 32];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) code[k] = ld_shared_v4(raw + (32 * k + lane) * 16);
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 s = ld_shared_v4(raw + 16 * D + 16 * i);
            h[2 * i] = pack_f16x2(__uint_as_float(s.x) * f, __uint_as_float(s.y) * f);
            h[2 * i + 1] = pack_f16x2(__uint_as_float(s.z) * f, __uint_as_float(s.w) * f);
        }
        const bool plain = live == 0xffffu && own == 0u;
        bool odd = false;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const int d = 32 * k + lane;
            const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = mul_f16x2(e4m3x2_to_f16x2((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu)), h[i]);
            if (!plain) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t bad = not_finite(o[i], 0x7c007c00u);
                    const uint32_t mine = ((own >> (2 * i)) & 1u ? 0xffffu : 0u) | ((own >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
                    const uint32_t key = ((live >> (2 * i)) & 1u ? 0xffffu : 0u) | ((live >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
                    odd |= (bad & mine) != 0u;
                    o[i] &= key & ~(bad & mine);
                }
            }
            st_shared_v4(dst + d * 16, make_uint4(o[0], o[1], o[2], o[3]));
            st_shared_v4(dst + kKeyBlocks * (D * 16) + d * 16, make_uint4(o[4], o[5], o[6], o[7]));
        }
        return odd;
    }
};

// 2^x as f16: 0 below its range, infinity above
__device__ __forceinline__ uint32_t f16_power(int x) {
    return x >= -14 ? (uint32_t)min(x + 15, 31) << 10 : x >= -24 ? 1u << (x + 24) : 0u;
}

template <int D>
struct Convert<D, PA_FP4_E2M1> {
    static constexpr int NB = D / 32;
    static constexpr int DEPTH = 23;           // (f16 holds every code times 2^-23 exactly)
    // The scale codes of a lane's four tokens, NB bytes each, plus 1, two to a word; 0 where they are no keys' or 255, which
    // is no number.  (Pairs of 16 bits have a maximum in one instruction, bytes have not.)
    struct Scales { uint32_t x[2 * NB]; };
    static __device__ __forceinline__ Scales scales(uint32_t raw, int rec, int keys, int lane) {
        const uint32_t at = raw + (lane >> 2) * rec + 8 * D + (lane & 3) * (4 * NB);
        const int n = keys - 4 * lane;
        Scales s;
        auto put = [&](int i, uint32_t x, uint32_t key) {
            s.x[2 * i] = ((x & 0x00ff00ffu) + 0x00010001u) & key & 0x00ff00ffu;
            s.x[2 * i + 1] = ((x >> 8 & 0x00ff00ffu) + 0x00010001u) & key & 0x00ff00ffu;
        };
        if constexpr (NB == 4) {
            const uint4 y = ld_shared_v4(at);
            put(0, y.x, n > 0 ? ~0u : 0u);
            put(1, y.y, n > 1 ? ~0u : 0u);
            put(2, y.z, n > 2 ? ~0u : 0u);
            put(3, y.w, n > 3 ? ~0u : 0u);
        } else {
            const uint2 y = ld_shared_v2(at);
            put(0, y.x, n > 1 ? ~0u : n > 0 ? 0xffffu : 0u);
            put(1, y.y, n > 3 ? ~0u : n > 2 ? 0xffffu : 0u);
        }
        return s;
    }
    static __device__ __forceinline__ int exponent(const Scales& s) {
        uint32_t m = s.x[0];
#pragma unroll
        for (int i = 1; i < 2 * NB; ++i) m = __vmaxu2(m, s.x[i]);
        return max((int)__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) - 1, 0);
    }
    // (a code of 0 counts as none: its values are 6 2^-127 at most)
    static __device__ __forceinline__ bool below(const Scales& s, int e) {
        uint32_t m = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) m = __vminu2(m, __vsub2(s.x[i], 0x00020002u));       // (none: passes to the top)
        return (int)min(m & 0xffffu, m >> 16) < e - 1;
    }
    // The largest code of each token of a wide tile, a byte a column; in the record its codes are against that, 127.
    static __device__ __forceinline__ void widen(uint32_t raw, int rec, uint32_t to, int, int, int lane) {
        const uint32_t at = raw + (lane >> 2) * rec + 8 * D + (lane & 3) * (4 * NB);
        uint32_t w = 0u;
#pragma unroll 1
        for (int t = 0; t < 4; ++t) {
            int top = 0;
            for (int b = 0; b < NB; ++b) {
                const int e = (int)code_at(at + t * NB + b);
                if (e != 255) top = max(top, e);
            }
            w |= (uint32_t)top << (8 * t);
            for (int b = 0; b < NB; ++b) {
                const int e = (int)code_at(at + t * NB + b);
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + t * NB + b), "r"(e == 255 ? e : max(e - top + 127, 0)) : "memory");
            }
        }
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 4 * lane), "r"(w) : "memory");
    }
    static __device__ __forceinline__ uint32_t code_at(uint32_t addr) {
        uint32_t v;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
        return v;
    }
    // the power of two of scale code e against the reference r (code 255: infinity)
    static __device__ __forceinline__ uint32_t power(uint32_t e, int r) { return e == 255u ? 0x7c00u : f16_power((int)e - r); }
    // Words read in an order of the lane's own, which begins at `by`, back in theirs.  (At head dim 128 a word's
    // bank hardly depends on which row it is of: read by all lanes in one order, eight of them would want the same
    // bank, 213 us instead of 190 for four sequences of 80000 tokens; at 64 there are four, 51.7 and 52.2 us
    // for 64 of 4096.)
    static __device__ __forceinline__ void turned_back(uint32_t (&x)[4], int by) {
        const bool one = by & 1, two = by & 2;
        const uint32_t a = one ? x[3] : x[0], b = one ? x[0] : x[1], c = one ? x[1] : x[2], d = one ? x[2] : x[3];
        x[0] = two ? c : a;
        x[1] = two ? d : b;
        x[2] = two ? a : c;
        x[3] = two ? b : d;
    }
    static __device__ __forceinline__ void keys(uint32_t raw, uint32_t dst, int ek, int lane) {
        const int slot = lane & 15, by = D == 128 ? (slot >> 1) & 3 : 0;
        uint32_t code[NB / 2][4], scale[NB / 2];
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
            const int w = 2 * k + (lane >> 4);
            scale[k] = code_at(raw + 8 * D + slot * NB + w);
#pragma unroll
            for (int c = 0; c < 4; ++c) code[k][c] = ld_shared_u32(raw + slot * (D / 2) + ((c + by) & 3) * (D / 8) + 4 * w);
        }
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
            const int w = 2 * k + (lane >> 4);
            const uint32_t e = power(scale[k], ek), h = e | e << 16;
            turned_back(code[k], by);
            uint32_t o[4][4];                                  // [c][piece]: dims 8 piece + 2 c, + 1
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                e2m1x8_to_f16x2x4(code[k][c], o[c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[c][i] = mul_f16x2(o[c][i], h);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st_shared_v4(dst + (4 * w + i) * (kKeyBlocks * 256) + slot * 16, make_uint4(o[0][i], o[1][i], o[2][i], o[3][i]));
        }
    }
    // `table`: 128 bytes of the warp's, a pair of tokens' powers of two for each 32 dims: [D / 32][8 pairs]
    static __device__ __forceinline__ bool values(uint32_t raw, uint32_t dst, uint32_t table, int rv, int lane, uint32_t live,
                                                  uint32_t own) {
        const int r = lane & 7, by = D == 128 ? r & 3 : 0;
        bool odd = false;
        uint32_t code[D / 64][4];
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) code[k][c] = ld_shared_u32(raw + ((4 * r + ((c + by) & 3)) * (D / 16) + 4 * k + (lane >> 3)) * 4);
        if (lane < 8 * NB) {
            const int t = 2 * r, b = lane >> 3;
            const uint32_t at = raw + 8 * D + t * NB + b;
            const uint32_t e0 = code_at(at), e1 = code_at(at + NB);
            uint32_t h = power(e0, rv) | power(e1, rv) << 16;
            const bool b0 = e0 == 255u && ((own >> t) & 1u), b1 = e1 == 255u && ((own >> (t + 1)) & 1u);
            odd = b0 || b1;
            if (b0 || !((live >> t) & 1u)) h &= 0xffff0000u;
            if (b1 || !((live >> (t + 1)) & 1u)) h &= 0xffffu;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(table + 4 * lane), "r"(h) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            const int mi = 4 * k + (lane >> 3);
            const uint4 lo = ld_shared_v4(table + mi / 2 * 32), hi = ld_shared_v4(table + mi / 2 * 32 + 16);
            const uint32_t h[2][4] = {{lo.x, lo.y, lo.z, lo.w}, {hi.x, hi.y, hi.z, hi.w}};
            turned_back(code[k], by);
            uint32_t o[4][4];                                  // [c][dh, half]: tokens 2 c + 8 half, + 1 of dim 16 mi + 8 dh + r
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                e2m1x8_to_f16x2x4(code[k][c], o[c]);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[c][x] = mul_f16x2(o[c][x], h[x & 1][c]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
                st_shared_v4(dst + (x & 1) * (D * 16) + (16 * mi + 8 * (x >> 1) + r) * 16,
                             make_uint4(o[0][x], o[1][x], o[2][x], o[3][x]));
        }
        __syncwarp();                                          // (the table's reads are done)
        return odd;
    }
};

// n arrivals on an mbarrier.
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// The same of E4M3 operands, 32 of K at a time.
__device__ __forceinline__ void umma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// N consecutive 32-bit columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]) {
    static_assert(N == 4 || N == 8 || N == 16 || N == 32);
    if constexpr (N == 4) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else if constexpr (N == 16) {
        tmem_st16(taddr, r);
    } else {
        tmem_st32(taddr, r);
    }
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N == 16 || N == 32);
    if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
    } else {
        tmem_ld32(taddr, r);
    }
}

// One element of a value as a number, from the pool.
template <int D, pa_dtype T>
__device__ __noinline__ float value_at(const char* rec, int slot, int d) {
    if constexpr (T == PA_BF16) {
        return bf16_lo_to_f32(*reinterpret_cast<const uint16_t*>(rec + ((d / 8) * kBlockTokens + slot) * 16 + (d % 8) * 2));
    } else if constexpr (T == PA_FP8_E4M3) {
        const uint32_t code = (uint8_t)rec[d * 16 + slot];
        // (what is asked is whether it is finite, and which infinity else)
        const float scale = *reinterpret_cast<const float*>(rec + 16 * D + 4 * slot);
        const float unit = (code & 0x7fu) == 0x7fu ? __int_as_float(0x7fc00000) : (code & 0x7fu) ? 1.f : 0.f;
        return (code & 0x80u ? -unit : unit) * scale;
    } else {
        const uint32_t e = (uint8_t)rec[8 * D + slot * (D / 32) + d / 32];
        if (e != 255u) return 0.f;
        const int at = ((4 * (d % 8) + (slot % 8) / 2) * (D / 16) + d / 16) * 4 + 2 * ((d % 16) / 8) + slot / 8;
        const uint32_t code = (uint8_t)rec[at] >> (4 * (slot & 1));
        return (code & 7u) == 0u ? __int_as_float(0x7fc00000) : __int_as_float(code & 8u ? 0xff800000 : 0x7f800000);
    }
}

// Wide tiles, whose scales lie further apart than operands of 16 bits against one reference hold: a column's own scales go
// on its score and on its probability, and a row has its O in a unit of its own, if need be, so that no row depends on
// the scales of keys that it does not see or that weigh nothing for it.  (64 sequences of 4096 tokens, 32 / 8 heads of 128,
// 8 nodes, all tiles wide: FP8 1360 us instead of 171, FP4 957 instead of 184.)

// A scale as 2^(e - 127) m, |m| from 1 to below 2; 0: m = 0; not finite: m is what it is.
struct Split {
    float m;
    int e;
};
__device__ __forceinline__ Split split_scale(uint32_t bits) {
    const float s = __uint_as_float(bits);
    if (!(fabsf(s) <= FLT_MAX)) return Split{s, 127};
    if (s == 0.f) return Split{0.f, 0};
    const bool small = fabsf(s) < FLT_MIN;
    const uint32_t b = __float_as_uint(small ? s * 0x1p64f : s);
    return Split{__uint_as_float((b & 0x807fffffu) | 0x3f800000u), (int)((b >> 23) & 0xffu) - (small ? 64 : 0)};
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
constexpr int kOwnUnits = -2;            // for `ev`, the exponent of the rows' unit of O: each has its own
// What a tile takes and leaves of a row: maximum, sum, ev; whether the waits went well.
struct WideRow {
    float m, l;
    int ev;
    bool ok;
};
// The softmax of a wide tile, the CTA's t-th, by the threads that share a row, with the same barriers as that of others;
// a function beside the loop over the tiles, which has to be short.  first: the piece's first tile; mrow: the row's mask words
// (null: no row), key0: its first key as a node; shift: what the row of q carries.
template <int D, pa_dtype T>
__device__ __noinline__ WideRow wide_tile(WideRow row, uint32_t sbase, uint32_t tmem, int t, bool first, const int32_t* mrow, int words,
                                          int key0, int nodes, int shift, float scale, float lift) {
    using L = Layout<D, T, 1>;
    constexpr int PARTS = Roles<T, 1>::PARTS, COLS = kKeys / PARTS, DP = D / PARTS;
    constexpr bool FP8 = T == PA_FP8_E4M3;
    const int warp = threadIdx.x >> 5, quarter = warp & 3, part = warp >> 2, lr = quarter * 32 + (threadIdx.x & 31);
    const int row_bar = 3 + quarter;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t scores = lanes + kColS + (t & 1) * kKeys + COLS * part, o = lanes + kColO + DP * part;
    const uint32_t table = sbase + L::WIDE + t % L::WIDE_TILES * L::WIDE_TILE;
    const uint2 e = ld_shared_v2(sbase + L::PASSED + (FP8 ? (t & 1) * L::PASS + kKeys * 4 : 8 * (t & 7)));
    const bool own = (e.y & kWideValues) != 0u;
    // column c's scale of values: its own, or the tile's power of two
    auto value_scale = [&](int c) {
        if (!own) return Split{1.f, (int)(e.y & 0xffu)};
        if constexpr (FP8) return split_scale(ld_shared_u32(table + 4 * (COLS * part + c)));
        else return Split{1.f, (int)ld_shared_u8(table + kKeys + COLS * part + c)};
    };
    auto exchange = [&](int at, float x) {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + at + 4 * (kTileRows * part + lr)), "f"(x) : "memory");
    };
    auto most = [&](int at, float x) {
#pragma unroll
        for (int k = 0; k < PARTS; ++k) x = fmaxf(x, __uint_as_float(ld_shared_u32(sbase + at + 4 * (kTileRows * k + lr))));
        return x;
    };
    // scores in log2 units, back to the TMEM; their maximum, and that of score + exponent of the value's scale
    const Split by = split_scale(__float_as_uint(fmaxf(scale, FLT_MIN)));
    const int ke = (int)(e.x & 0xffu) - 254 - shift + by.e;
    float mx = -INFINITY, ux = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 16) {
        uint32_t r[16];
        tmem_ld(scores + c, r);
        tmem_wait_ld();
        // 16 columns: the keys in their order; FP8: eight of one half of each block's slots, then of the next block's
        uint32_t see = 0u;
        if (mrow) {
            const int col = COLS * part + c;
            if constexpr (FP8) {
                const uint32_t w = seen_word(mrow, words, key0 + (col & 63) * 2, nodes) >> (col >> 6) * 8;
                see = (w & 0xffu) | (w >> 8 & 0xff00u);
            } else {
                see = seen_word(mrow, words, key0 + col, nodes);
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            // (FP8's keys: the scale over the power of two in e)
            const Split s = FP8 ? split_scale(ld_shared_u32(sbase + L::PASSED + (t & 1) * L::PASS + 4 * (COLS * part + c + k)))
                                : Split{1.f, own ? (int)ld_shared_u8(table + COLS * part + c + k) : 127};
            // (two powers of two: past fp32's range only where the score is)
            const int n = max(-252, min(ke + s.e - 127, 252));
            float x = __uint_as_float(r[k]) * (s.m * by.m) * exp2i(n / 2) * exp2i(n - n / 2);
            x = (see >> k) & 1u ? x : -INFINITY;
            r[k] = __float_as_uint(x);
            const Split v = value_scale(c + k);
            mx = fmaxf(mx, x);
            if (v.m != 0.f && fabsf(v.m) <= FLT_MAX) ux = fmaxf(ux, x + (float)v.e);
        }
        tmem_st16(scores + c, r);
    }
    tmem_wait_st();
    // and the largest element of O
    float ox = 0.f;
    if (!first) {
        row.ok = warp_wait(sbase + L::BAR + 8 * kPVDone, (t - 1) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DP && row.ok; c += 16) {
            uint32_t x[16];
            tmem_ld(o + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) ox = fmaxf(ox, fabsf(__uint_as_float(x[k])));
        }
    }
    named_bar_or(row_bar, 32 * PARTS, true);
    exchange(L::ROWS, mx);
    exchange(L::TOPS, ux);
    exchange(L::LARGEST, ox);
    named_bar_sync(row_bar, 32 * PARTS);
    mx = most(L::ROWS, mx);
    ux = most(L::TOPS, ux);
    ox = most(L::LARGEST, ox);
    const float was = row.m;
    if (mx > was) {
        row.m = mx;
        row.l *= fast_exp2(was - mx);
    }
    // O's unit over the maximum.  V's reference, while that holds what is in O and what the tile adds (2^-12 of it at least,
    // so that f16's smallest step is 2^-20 of the largest product), for all rows, as the next tile takes it then; else for
    // each row what this tile adds at most, unless what is in O would pass 2^100.
    const uint32_t units = sbase + L::UNITS + 4 * (kTileRows * part + lr);
    const float base = row.m == -INFINITY ? 0.f : row.m;
    const int reference = own ? (int)(e.x >> 8) : (int)(e.y & 0xffu);
    const float was_unit = (float)(row.ev == kOwnUnits ? (int)ld_shared_u32(units) : row.ev);
    const float had = ox > 0.f ? was - base + was_unit : -INFINITY, adds = ux - base, over = adds - (float)reference;
    const float in_o = had + (float)((int)(__float_as_uint(ox) >> 23) - 127), there = in_o - (float)reference;
    const bool fits = !mrow || (there <= 40.f && (there >= -40.f || adds >= in_o + 40.f || in_o == -INFINITY) &&
                                over <= 7.f && (over >= -12.f || adds <= in_o - 40.f || adds == -INFINITY));
    int unit = reference;
    row.ev = unit;
    if (!__all_sync(0xffffffffu, fits)) {
        row.ev = kOwnUnits;
        unit = (int)fminf(fmaxf(ceilf(fmaxf(adds, in_o - 100.f)), 1.f), 254.f);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(units), "r"(unit) : "memory");
    }
    if (!first) {
        // (in two steps, as a power of two alone may be out of range)
        const float by2 = had - (float)unit, near = fmaxf(-120.f, fminf(by2, 120.f)), part1 = fast_exp2(near), part2 = fast_exp2(by2 - near);
#pragma unroll 1
        for (int c = 0; c < DP && row.ok; c += 16) {
            uint32_t x[16];
            tmem_ld(o + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * part1 * part2);
            tmem_st(o + c, x);
        }
    }
    named_bar_sync(row_bar, 32 * PARTS);                              // (the maxima are read)
    if (!row.ok) return row;
    // the probabilities times their values' scales, as f16 against O's unit
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 16) {
        uint32_t r[16], w[8];
        tmem_ld(scores + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float x = __uint_as_float(r[k]) - base + lift;
            const Split v = value_scale(c + k);
            sum += fast_exp2(x);
            r[k] = __float_as_uint(fast_exp2(x + (float)(v.e - unit)) * v.m);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_f16x2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
        tmem_st(scores + c / 2, w);
    }
    row.l += sum;
    return row;
}

template <int D, pa_dtype T, int SW>
__global__ void __launch_bounds__(Roles<T, SW>::THREADS, 1) tree_tc_kernel(const __grid_constant__ TParams p) {
    using L = Layout<D, T, SW>;
    using W = Roles<T, SW>;
    constexpr bool RAW = L::RAW, NAT = L::NAT;
    constexpr int TILE = L::TILE, KTILE = L::KTILE, KSTAGE = L::KSTAGE, KST = L::KST, VST = L::VST, REC = L::REC;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + L::BAR + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < KST; ++i) {
            mbar_init(bar(kKFull + i), NAT ? 1 : RAW ? kKeyBlocks : W::FEEDS);
            mbar_init(bar(kKEmpty + i), 1);
        }
#pragma unroll
        for (int i = 0; i < VST; ++i) {
            mbar_init(bar(kVFull + i), RAW ? kKeyBlocks : 1);
            mbar_init(bar(kVEmpty + i), 1);
        }
#pragma unroll
        for (int i = 0; i < L::RST; ++i) {
            mbar_init(bar(kRFull + i), 1);
            mbar_init(bar(kREmpty + i), kKeyBlocks + 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kSFull + i), RAW ? 2 : 1);      // (RAW: the MMA warp passes the exponents on)
            mbar_init(bar(kPFull + i), 4 * W::PARTS);
            mbar_init(bar(kODone + i), 2);
            mbar_init(bar(kQFull + i), 4 * W::PARTS);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(kXFull + i), 1);
            mbar_init(bar(kXEmpty + i), W::READERS);
        }
        mbar_init(bar(kPVDone), 1);
        mbar_init(bar(kOFree), W::SOFT);
        mbar_init(bar(kDone), 1);
        if (RAW) {
            for (int i = 0; i < 4; ++i) mbar_init(bar(kEFull + i), 1);
            for (int i = 0; i < 2; ++i) *reinterpret_cast<volatile int*>(smem + L::GONE + 4 * i) = INT32_MAX;
        }
        fence_proxy_async_smem();
    }
    // lengths, tables, masks, queries and pools may be the previous kernels' output
    grid_dependency_wait();
    grid_launch_dependents();
    int32_t flag = 0;                                     // (under way with the lengths)
    if (threadIdx.x == 0 && p.err) flag = *reinterpret_cast<const volatile int32_t*>(p.err);
    Walk walk;
    {
        const Line line = tree_locate<W::THREADS, kKeys>(
            p, reinterpret_cast<long long*>(smem + L::Q), blockIdx.x == 0,
            [&](const Line& l) { return (int)blockIdx.x < l.ctas ? l.begin(blockIdx.x) : l.total; }, walk.c);
        const bool any = (int)blockIdx.x < line.ctas && line.total > 0;
        walk.left = any ? line.begin(blockIdx.x + 1) - line.begin(blockIdx.x) : 0;
        if (walk.left <= item_cost(kKeys) - walk.c.at) walk.left = 0;            // (ends before a first tile)
        // (said whether or not the call goes on, by the last thread, which has the least to do)
        if (threadIdx.x == W::THREADS - 1) say_joint(p, line, walk.c, blockIdx.x, any);
    }
    if (threadIdx.x == 0) *reinterpret_cast<Walk*>(smem + L::FIRST) = walk;
    // (the same for all threads, and the search's scratch is free)
    if (__syncthreads_or(flag & PA_DEV_ERR_TIMEOUT) || walk.left == 0) return;
    // the ic-th piece of the CTA
    auto piece = [&](int ic, Piece& x) -> bool {
        if (!warp_wait(bar(kXFull + ic % kPieces), (ic / kPieces) & 1)) return false;
        const uint32_t at = sbase + L::RECORDS + (ic % kPieces) * 32;
        const uint4 a = ld_shared_v4(at), b = ld_shared_v4(at + 16);
        x.j0 = (int)a.x;
        x.n = (int)a.y;
        x.tokens = (int)a.z;
        x.qrow = (int)a.w;
        x.start = (int)b.x;
        x.nodes = (int)b.y;
        x.s = (int)b.z;
        x.h = (int)(b.w & 0x7fffffffu);
        x.whole = b.w >> 31;
        return true;
    };
    auto piece_done = [&](int ic) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kXEmpty + ic % kPieces));
    };

    if (warp >= W::SOFT) {
    if (warp == W::COPY) {
        // ------------------------------------------------------------ bulk copies
        // Lane b block b.  bf16: V tiles; FP8: K tiles and V's records; FP4: the records, K's and V's of
        // a tile one after the other.
        const uint64_t pol = l2_policy_evict_first();
        constexpr int ST = RAW ? L::RST : VST, PER = RAW ? 2 : 1;
        const int full0 = RAW ? kRFull : kVFull, empty0 = RAW ? kREmpty : kVEmpty;
        bool ok = true;
        int u = 0, uk = 0;                            // stages filled so far (K's own: FP8)
        Piece ahead = walk.piece(p);
        auto put = [&](int ic) {
            if (ic >= kPieces) ok = ok && warp_wait(bar(kXEmpty + ic % kPieces), (ic / kPieces - 1) & 1);
            if (ok && lane == 0) {
                const uint32_t at = sbase + L::RECORDS + (ic % kPieces) * 32;
                st_shared_v4(at, make_uint4(ahead.j0, ahead.n, ahead.tokens, ahead.qrow));
                st_shared_v4(at + 16, make_uint4(ahead.start, ahead.nodes, ahead.s, (uint32_t)ahead.h | (ahead.whole ? 1u << 31 : 0u)));
                mbar_arrive(bar(kXFull + ic % kPieces));
            }
            __syncwarp();
        };
        put(0);
        for (int ic = 0; ok && ahead.n > 0; ++ic) {
            const Piece x = ahead;
            walk.next(p);
            ahead = walk.piece(p);
            put(ic + 1);
            Table table(p, x, lane);
            for (int i = 0; ok && i < x.n; ++i) {
                const int32_t blk = table.block(p, i);
                const bool mine = blk >= 0 && lane < kKeyBlocks;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * REC;
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const bool to_k = NAT && k == 0;
                    int& at = to_k ? uk : u;
                    const int ring = to_k ? KST : ST, st = at % ring;
                    const uint32_t full = bar((to_k ? kKFull : full0) + st);
                    if (at >= ring) {
                        ok = warp_wait(bar((to_k ? kKEmpty : empty0) + st), (at / ring - 1) & 1);
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        fence_proxy_async_smem();
                        mbar_arrive_expect_tx(full, bytes);
                    }
                    __syncwarp();
                    if (mine) {
                        const char* pool = RAW && k == 0 ? p.k_pool : p.v_pool;
                        const uint32_t dst = to_k ? L::K + st * KSTAGE + lane * REC : RAW ? L::R + st * L::HALF + lane * REC : L::V + st * KTILE + lane * TILE;
                        bulk_g2s(sbase + dst, pool + ((size_t)blk * p.Hkv + x.h) * (size_t)REC, REC, full, pol);
                    }
                    ++at;
                }
            }
        }
        if (!ok && lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        // before the CTA ends, every copy has landed
        if (lane == 0) {
            for (int f = max(0, u - ST); f < u; ++f) mbar_wait_bounded(bar(full0 + f % ST), (f / ST) & 1, kLandNs);
            for (int f = max(0, uk - KST); f < uk; ++f) mbar_wait_bounded(bar(kKFull + f % KST), (f / KST) & 1, kLandNs);
        }
    } else if (warp == W::MMA) {
        // ------------------------------------------------------------ MMA issue
        // MMAs execute in issue order, so S(t + 2) (or S_h(t + 1) with two row tiles) overwrites
        // P(t)'s columns only after P V(t) has read them.
        tmem_alloc<512>(sbase + L::SLOT);
        tc_fence_before();
        named_bar_sync(2, 32 * (W::SOFT + 1));
        tc_fence_after();
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::SLOT);
        constexpr uint32_t idS = idesc(RAW, NAT ? kKeys / 2 : kKeys, 0), idO = idesc(RAW, D, RAW ? 0 : 1);
        bool ok = true;
        int t0 = 0;
        for (int ic = 0; ok; ++ic) {
            Piece x;
            ok = piece(ic, x);
            if (!ok || x.n == 0) break;
            const int n = x.n, nblk = x.blocks();
            bool odd = false;
            auto issue_s = [&](int hh, int i) {
                const int t = t0 + i, buf = SW == 2 ? hh : t & 1;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = umma_desc(sbase + L::Q + hh * L::QTILE, 2048, 128);
                    const uint32_t dcol = tmem + kColS + (uint32_t)(buf * kKeys), qcol = tmem + kColQ + (uint32_t)((ic & 1) * (D / 2));
                    if constexpr (NAT) {
                        // eight slots of a block are eight rows of the operand, 16 dims each: the blocks' first
                        // eight, a record apart, are one operand of 64 rows, their last eight another
                        const uint64_t kd = umma_desc(sbase + L::K + (t % KST) * KSTAGE, 256, REC);
#pragma unroll
                        for (int m = 0; m < D / 8; ++m) {              // [slots' half][part of q][32 dims]
                            const int hf = m / (D / 16), a = m % (D / 16), ks = a % (D / 32);
                            umma_ts_f8(dcol + 64 * hf, qcol + 8 * a, kd + (uint64_t)((hf * 128 + ks * 512) >> 4), idS, a > 0);
                        }
                    } else {
                        const uint64_t kd = umma_desc(sbase + L::K + (t % KST) * KSTAGE, kKeyBlocks * 256, 128);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint64_t kk = kd + (uint64_t)((ks * 2 * kKeyBlocks * 256) >> 4);
                            if (SW == 1) umma_ts(dcol, qcol + 8 * ks, kk, idS, ks > 0);
                            else umma_ss(dcol, qd + (uint64_t)(ks * 256), kk, idS, ks > 0);
                        }
                    }
                    umma_commit(bar(kSFull + buf));
                    if constexpr (RAW && !NAT) {
                        st_shared_v2(sbase + L::PASSED + 8 * (t & 7), ld_shared_v2(sbase + L::EXPS + 8 * (t & 7)));
                        mbar_arrive(bar(kSFull + buf));
                    }
                }
                __syncwarp();
                if constexpr (NAT) {
                    // the columns' scales in their order, against the largest's power of two (so that no score
                    // overflows that does not with the row's factor): a lane has four slots of a block
                    const uint32_t to = sbase + L::PASSED + buf * L::PASS, at = sbase + L::K + (t % KST) * KSTAGE;
                    const auto scales = Convert<D, T>::scales(at, REC, x.end() - (x.j0 + i) * kKeys, lane);
                    int ek = Convert<D, T>::exponent(scales);
                    // (too far apart for products in fp32: as they are)
                    const bool wide = __any_sync(0xffffffffu, Convert<D, T>::below(scales, ek - 60));
                    if (wide) ek = 127;
                    const uint4 sk = ld_shared_v4(at + (lane >> 2) * REC + 16 * D + (lane & 3) * 16);
                    const float f = exp2i(127 - ek);
                    st_shared_v4(to + ((lane >> 1) & 1) * 256 + (lane >> 2) * 32 + (lane & 1) * 16,
                                 make_uint4(__float_as_uint(__uint_as_float(sk.x) * f), __float_as_uint(__uint_as_float(sk.y) * f),
                                            __float_as_uint(__uint_as_float(sk.z) * f), __float_as_uint(__uint_as_float(sk.w) * f)));
                    ok = warp_wait(bar(kEFull + (t & 3)), (t >> 2) & 1);
                    if (lane == 0) {
                        const uint2 e = ld_shared_v2(sbase + L::EXPS + 8 * (t & 7));
                        st_shared_v2(to + kKeys * 4, make_uint2((uint32_t)ek | (e.x & 0xff00u), e.y | (wide ? kWideKeys : 0u)));
                    }
                    __syncwarp();
                    if (elect_one()) mbar_arrive(bar(kSFull + buf));
                    __syncwarp();
                }
            };
            auto k_ready = [&](int i) { ok = warp_wait(bar(kKFull + (t0 + i) % KST), ((t0 + i) / KST) & 1); };
            auto k_free = [&](int i) {
                if (elect_one()) umma_commit(bar(kKEmpty + (t0 + i) % KST));
                __syncwarp();
            };
            auto issue_pv = [&](int hh, int i) {
                const int t = t0 + i, st = t % VST, buf = SW == 2 ? hh : t & 1;
                ok = SW == 2 ? warp_wait(bar(kPFull + hh), t & 1) : warp_wait(bar(kPFull + buf), (t >> 1) & 1);
                if (!ok) return;
                if (i == 0 && hh == 0 && ic > 0) {
                    ok = warp_wait(bar(kOFree), (ic - 1) & 1);            // the last piece's O is read
                    if (!ok) return;
                }
                const int tok0 = (x.j0 + i) * kKeys, nb = min(kKeyBlocks, nblk - (x.j0 + i) * kKeyBlocks);
                if (hh == 0) {
                    ok = warp_wait(bar(kVFull + st), (t / VST) & 1);
                    if (!ok) return;
                    if constexpr (RAW) {
                        const uint2 o = ld_shared_v2(sbase + L::SEEN + 8 * (t & 7));
                        odd |= (o.x | o.y) != 0u;
                    } else if (tok0 + nb * kBlockTokens > x.start) {
                        // slots past the last key may hold anything: zeros; values of the tree's own
                        // tokens that are no finite numbers too (looked for in all of its blocks)
                        const int from = max(x.start - tok0, 0), to = x.end() - tok0;
                        uint8_t* const vt = smem + L::V + st * KTILE;
                        constexpr int PIECES = (D / 8) * kBlockTokens;                 // of a block
                        if (to < nb * kBlockTokens) {
                            uint8_t* const last = vt + (nb - 1) * TILE;
                            for (int e = lane; e < PIECES; e += 32)
                                if ((nb - 1) * kBlockTokens + e % kBlockTokens >= to)
                                    *reinterpret_cast<uint4*>(last + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                            __syncwarp();
                        }
                        uint32_t top = 0u;                              // largest magnitudes, 16 bits each
                        for (int b = from / kBlockTokens; b < nb; ++b) {
#pragma unroll
                            for (int e = 0; e < PIECES / 32; ++e) {
                                const uint4 v = *reinterpret_cast<const uint4*>(vt + b * TILE + (32 * e + lane) * 16);
                                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                             __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                            }
                        }
                        if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u)) {
                            odd = true;
                            for (int e = from / kBlockTokens * PIECES + lane; e < nb * PIECES; e += 32) {
                                const int key = e / PIECES * kBlockTokens + e % kBlockTokens;
                                if (key < from) continue;
                                const uint4 v = *reinterpret_cast<const uint4*>(vt + e * 16);
                                const uint32_t m = 0x7f807f80u;
                                *reinterpret_cast<uint4*>(vt + e * 16) =
                                    make_uint4(v.x & ~not_finite(v.x, m), v.y & ~not_finite(v.y, m), v.z & ~not_finite(v.z, m), v.w & ~not_finite(v.w, m));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t pcol = tmem + kColS + (uint32_t)(buf * kKeys), ocol = tmem + kColO + (uint32_t)(hh * kKeys);
                    // bf16: a block as stored, [D/8][16 slots][8 dims]; else [2 groups][D/8][8 dims][8 tokens], FP8's
                    // groups the blocks' first eight slots, then their last eight, as the columns of S are
                    const uint64_t vd = RAW ? umma_desc(sbase + L::V + st * KTILE, D * 16, 128)
                                            : umma_desc(sbase + L::V + st * KTILE, 128, 256);
                    const uint32_t more = i > 0 ? 1u : 0u;
                    constexpr int PB = kKeyBlocks / W::PARTS;           // each part of the rows' threads begins at its own columns
                    auto pv = [&](int b) {
                        umma_ts(ocol, pcol + kKeys / W::PARTS * (b / PB) + 8 * (b % PB), vd + (uint64_t)((b * TILE) >> 4), idO, b > 0 ? 1u : more);
                    };
                    if (nb == kKeyBlocks) {
#pragma unroll
                        for (int b = 0; b < kKeyBlocks; ++b) pv(b);
                    } else {
                        for (int b = 0; b < kKeyBlocks; ++b)
                            if ((NAT ? 2 * (b % 4) : b) < nb) pv(b);
                    }
                    if (hh == SW - 1) umma_commit(bar(kVEmpty + st));
                    if (SW == 1) umma_commit(bar(kPVDone));
                }
                __syncwarp();
                if (i == n - 1) {
                    odd = __any_sync(0xffffffffu, odd);
                    if (elect_one()) {
                        umma_commit(bar(kODone + hh));
                        if (hh == 0) *reinterpret_cast<volatile uint32_t*>(smem + L::ODD + 4 * (ic & 1)) = odd;
                        mbar_arrive(bar(kODone + hh));
                    }
                    __syncwarp();
                }
            };
            if constexpr (SW == 1) {
                ok = warp_wait(bar(kQFull + (ic & 1)), (ic >> 1) & 1);
                for (int i = 0; ok && i < n + 2; ++i) {
                    // S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ...
                    if (i >= 2) issue_pv(0, i - 2);
                    if (ok && i < n) {
                        k_ready(i);
                        if (!ok) break;
                        issue_s(0, i);
                        k_free(i);
                    }
                }
            } else {
                // S_a(0) S_b(0) | PV_a(0) S_a(1) PV_b(0) S_b(1) | ...
                ok = warp_wait(bar(kQFull), ic & 1);
                if (ok) k_ready(0);
                if (ok) issue_s(0, 0);
                if (ok) ok = warp_wait(bar(kQFull + 1), ic & 1);
                if (ok) {
                    issue_s(1, 0);
                    k_free(0);
                }
                for (int i = 0; ok && i < n; ++i) {
                    const bool more = i + 1 < n;
                    issue_pv(0, i);
                    if (ok && more) {
                        k_ready(i + 1);
                        if (ok) issue_s(0, i + 1);
                    }
                    if (ok) issue_pv(1, i);
                    if (ok && more) {
                        issue_s(1, i + 1);
                        k_free(i + 1);
                    }
                }
            }
            t0 += n;
            piece_done(ic);
        }
        if (!ok && lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        // nothing may still be running on the tensor cores when the TMEM is freed
        if (elect_one()) umma_commit(bar(kDone));
        __syncwarp();
        mbar_wait_bounded(bar(kDone), 0, kLandNs);
    } else if (RAW && warp >= W::LEAD && warp < W::LEAD + W::LEADS) {
        // ------------------------------------------------------------ the conversions' lead
        // One warp for the keys, one for the values waits for a tile's records and for its place and lets
        // eight warps go at a named barrier, so that they do not poll (28 polling warps took half of
        // the issue slots).  The first also finds the tile's largest K scale, and V's reference: the
        // piece's first, moved to a tile's largest that is 2^6 above or below it.  O, up to 2^42, moves with it, so
        // not by more than 2^60.  A tile with scales too far from it is a wide one.
        if constexpr (RAW) {
            using C = Convert<D, T>;
            const bool for_v = NAT || warp > W::LEAD;
            bool ok = true;
            int t = 0;
            // (two barriers in turn: a tile's place is free when the conversions two tiles before are done, so that
            // their barrier is too)
            static_assert(VST == 2 && (NAT || KST == 2), "a tile's place is that of two tiles before");
            const int go = 7 + 2 * for_v;
            const uint32_t gone = sbase + L::GONE + 4 * for_v, done = bar(for_v ? kVFull : kKFull);
            for (int ic = 0; ok; ++ic) {
                Piece x;
                ok = piece(ic, x);
                if (!ok) conversions_leave(t, gone, done, go);
                if (!ok || x.n == 0) break;
                int rv = 127, top = 0, low = 255;         // (of references: V's, the highest, the lowest; top 0: none yet)
                for (int i = 0; i < x.n; ++i, ++t) {
                    const int uk = 2 * t, uv = NAT ? t : 2 * t + 1, rk = uk % L::RST, rs = uv % L::RST;
                    const int keys = x.end() - (x.j0 + i) * kKeys;
                    if (NAT || !for_v) {
                        const uint32_t kraw = sbase + L::R + rk * L::HALF, vraw = sbase + L::R + rs * L::HALF;
                        int ek = 0;
                        bool far = false;
                        if (!NAT) {
                            ok = warp_wait(bar(kRFull + rk), (uk / L::RST) & 1);
                            const auto scales = C::scales(kraw, REC, keys, lane);
                            ek = C::exponent(scales);
                            far = C::below(scales, ek - C::DEPTH);
                        }
                        ok = ok && warp_wait(bar(kRFull + rs), (uv / L::RST) & 1);
                        const auto scales = C::scales(vraw, REC, keys, lane);
                        const int ev = C::exponent(scales);
                        if (ev > 0 && (top == 0 || ev > rv + 6 || ev < rv - 6)) {
                            if (max(top, ev) - min(low, ev) > 60 && top > 0) {
                                far = true;
                            } else {
                                rv = ev;
                                top = max(top, ev);
                                low = min(low, ev);
                            }
                        }
                        const bool wide = __any_sync(0xffffffffu, far || C::below(scales, rv - C::DEPTH));
                        if (ok && wide) {
                            const uint32_t to = sbase + L::WIDE + t % L::WIDE_TILES * L::WIDE_TILE;
                            const int ctx = x.start - (x.j0 + i) * kKeys;
                            if (!NAT) C::widen(kraw, REC, to, keys, ctx, lane);
                            C::widen(vraw, REC, NAT ? to : to + kKeys, keys, ctx, lane);
                            fence_proxy_async_smem();                // (before the next copies to the records' places)
                            __syncwarp();
                        }
                        if (ok && lane == 0) {
                            st_shared_v2(sbase + L::EXPS + 8 * (t & 7),
                                         wide ? make_uint2(127u | (uint32_t)rv << 8, 127u | kWideValues) : make_uint2((uint32_t)ek, (uint32_t)rv));
                            mbar_arrive(bar(kEFull + (t & 3)));
                            if (!NAT) mbar_arrive(bar(kREmpty + rk));
                            mbar_arrive(bar(kREmpty + rs));
                        }
                    } else {
                        ok = warp_wait(bar(kEFull + (t & 3)), (t >> 2) & 1);
                    }
                    if (for_v) {
                        if (t >= VST) ok = ok && warp_wait(bar(kVEmpty + t % VST), (t / VST - 1) & 1);
                    } else {
                        if (t >= KST) ok = ok && warp_wait(bar(kKEmpty + t % KST), (t / KST - 1) & 1);
                    }
                    if (!ok) {
                        conversions_leave(t, gone, done, go);
                        break;
                    }
                    __syncwarp();
                    named_bar_arrive(go + (t & 1), 32 * (kKeyBlocks + 1));
                }
                piece_done(ic);
            }
            if (!ok && lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        }
    } else if (warp < W::FEED + W::FEEDS) {
        const int f = warp - W::FEED;
        if constexpr (RAW) {
            // -------------------------------------------------------- conversions, one block of every
            // tile: warps 0 .. 7 its keys, 8 .. 15 its values (so that the keys of a tile do not wait
            // for the values of the one before)
            using C = Convert<D, T>;
            const int b = f % kKeyBlocks;
            const bool for_v = NAT || f >= kKeyBlocks;
            const uint32_t smem_r = sbase + L::R;
            bool ok = true;
            int t = 0;
            for (int ic = 0; ok; ++ic) {
                Piece x;
                ok = piece(ic, x);
                if (!ok) {
                    conversions_leave(t, sbase + L::GONE + 4 * for_v, 0u, 7 + 2 * for_v);
                    if (lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
                }
                if (!ok || x.n == 0) break;
                const int end = x.end();
                for (int i = 0; i < x.n; ++i, ++t) {
                    // (stages of K and V in turn)
                    const int uk = 2 * t, uv = NAT ? t : 2 * t + 1, rk = uk % L::RST, rs = uv % L::RST, st = for_v ? t % VST : t % KST;
                    const uint32_t vraw = smem_r + rs * L::HALF;
                    const int tok0 = (x.j0 + i) * kKeys, first = tok0 + b * kBlockTokens;
                    named_bar_sync(7 + 2 * for_v + (t & 1), 32 * (kKeyBlocks + 1));
                    ok = *reinterpret_cast<volatile int*>(smem + L::GONE + 4 * for_v) > t;
                    if (!ok) break;
                    mbar_test(bar(kRFull + (for_v ? rs : rk)), ((for_v ? uv : uk) / L::RST) & 1);     // (the copies are seen)
                    const uint2 e = ld_shared_v2(sbase + L::EXPS + 8 * (t & 7));
                    const int rv = (int)(e.y & 0xffu);
                    if (for_v) {
                        bool odd = false;
                        // (FP8: an odd last block has the next one's zeros beside it)
                        if (first < end || (NAT && (b & 1) && first - kBlockTokens < end)) {
                            const int keys = min(max(end - first, 0), kBlockTokens), ctx = min(max(x.start - first, 0), kBlockTokens);
                            const uint32_t live = (1u << keys) - 1u, own = live & ~((1u << ctx) - 1u);
                            odd = C::values(vraw + b * REC, sbase + L::V + st * KTILE + b * (NAT ? D * 16 : TILE), sbase + L::TABLE + b * 128, rv, lane,
                                            live, own);
                        }
                        odd = __any_sync(0xffffffffu, odd);
                        if (lane == 0) *reinterpret_cast<volatile uint8_t*>(smem + L::SEEN + 8 * (t & 7) + b) = odd;
                    } else if constexpr (!NAT) {
                        if (first < end) C::keys(smem_r + rk * L::HALF + b * REC, sbase + L::K + st * KTILE + b * 256, (int)(e.x & 0xffu), lane);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar((for_v ? kVFull : kKFull) + st));
                        mbar_arrive(bar(kREmpty + (for_v ? rs : rk)));
                    }
                }
                piece_done(ic);
            }
        } else {
            // -------------------------------------------------------- K's pieces
            // Tiles are published in order, each as soon as its copies have landed; a new one is issued
            // whenever its stage is free, two ahead at most.
            static_assert(RAW || KST <= 3, "the landing waits below cover up to two newer tiles");
            constexpr int PER = kBlockTokens * (D / 8) / (32 * W::FEEDS);     // pieces per thread and block
            const uint64_t pol = l2_policy_evict_first();
            const int kt = f * 32 + lane;
            bool ok = true;
            int t0 = 0;
            for (int ic = 0; ok; ++ic) {
                Piece x;
                ok = piece(ic, x);
                if (!ok || x.n == 0) break;
                const int n = x.n;
                Table table(p, x, lane);
                int next = 0;
                auto issue = [&]() {
                    const uint32_t dst = sbase + L::K + (t0 + next) % KST * KTILE;
                    const int32_t blk = table.block(p, next);
#pragma unroll
                    for (int b = 0; b < kKeyBlocks; ++b) {
                        const int32_t bb = __shfl_sync(0xffffffffu, blk, b);
                        if (bb < 0) continue;
                        const char* src = p.k_pool + ((size_t)bb * p.Hkv + x.h) * (size_t)TILE;
#pragma unroll
                        for (int u = 0; u < PER; ++u) {
                            const int piece = u * 32 * W::FEEDS + kt;
                            cp_async_16(dst + (piece >> 4) * (kKeyBlocks * 256) + b * 256 + (piece & 15) * 16, src + piece * 16, pol);
                        }
                    }
                    cp_async_commit();
                    ++next;
                };
                auto free_now = [&](int t) {
                    return t < KST || __all_sync(0xffffffffu, mbar_test(bar(kKEmpty + t % KST), (t / KST - 1) & 1));
                };
                for (int pub = 0; pub < n; ++pub) {
                    while (next < n && next - pub < 2 && free_now(t0 + next)) issue();
                    if (next == pub) {
                        ok = warp_wait(bar(kKEmpty + (t0 + next) % KST), ((t0 + next) / KST - 1) & 1);
                        if (!ok) break;
                        issue();
                    }
                    if (next - pub - 1 >= 1) cp_async_wait<1>();
                    else cp_async_wait<0>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kKFull + (t0 + pub) % KST));
                }
                t0 += n;
                piece_done(ic);
            }
            if (!ok && lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
            cp_async_wait<0>();
        }
    }
    } else {
    // ---------------------------------------------------------------- softmax, a row to PARTS threads
    // Warps w, w + 4, .. of a row tile's reach the TMEM lanes 32 (w % 4) .. and share its rows, each with
    // its part of the tile's columns (less code and waiting than a warp that takes them all).  They agree
    // on the row's maximum through shared memory where it rises.
    constexpr int PARTS = W::PARTS, COLS = kKeys / PARTS, NC = COLS / 32, DP = D / PARTS;
    const int quarter = warp & 3, part = (warp >> 2) % PARTS, h = warp / (4 * PARTS);
    const int lr = quarter * 32 + lane, row = h * kTileRows + lr;
    const int tl = row / p.G, g = row - tl * p.G;                     // token of the row tile, query head
    const uint32_t lanes_at = (uint32_t)(32 * quarter) << 16;
    const int row_bar = 3 + 4 * h + quarter;                          // the named barrier of the warps with the same rows
    float* const shared_row = reinterpret_cast<float*>(smem + L::ROWS) + (h * PARTS) * kTileRows + lr;    // [part]
    const float scale = fabsf(p.scale_log2);
    // a negative scale is applied as |scale| to -q, so that the row's maximum is that of the unscaled scores
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    constexpr int QB = D / 8;
    // A warp without rows only keeps the barriers going.
    auto busy = [&](const Piece& x) { return row - lane < x.tokens * p.G; };
    // row r of the row tile
    auto q_of = [&](const Piece& x, int token, int head) {
        return static_cast<const uint16_t*>(p.q) + ((size_t)(x.qrow + token) * p.Hq + (size_t)x.h * p.G + head) * D;
    };
    uint32_t tmem = 0u;
    int shift = 0;                                                    // (log2) of what the row of q carries
    // One row tile: the rows of the warps come to shared memory by whole rows (a thread that loads its
    // own row touches 32 lines at a time: 12000 clocks a piece), 16-byte piece u of row r at place u ^ r % 8,
    // and each goes through registers into the TMEM, columns of the piece's parity, a part of them by
    // each of the row's threads.
    auto stage_q = [&](const Piece& x) {
        if (busy(x)) {
#pragma unroll 1
            for (int k = part; k < QB; k += PARTS) {
                const int e = 32 * k + lane, r = 32 * quarter + e / QB, u = e % QB, token = r / p.G;
                const uint32_t to = sbase + L::Q + r * (2 * D) + (uint32_t)((u ^ (r & 7)) * 16);
                if (token < x.tokens) cp_async_16(to, q_of(x, token, r - token * p.G) + 8 * u);
                else st_shared_v4(to, make_uint4(0u, 0u, 0u, 0u));
            }
        }
        cp_async_commit();
    };
    auto put_q = [&](const Piece& x, int ic) -> int {
        float f = 1.f;
        int shift = 0;
        cp_async_wait<0>();
        if (busy(x)) {
            named_bar_sync(row_bar, 32 * PARTS);                      // (the rows)
            auto at = [&](int u) { return ld_shared_v4(sbase + L::Q + lr * (2 * D) + (uint32_t)(((part * (DP / 8) + u) ^ (lr & 7)) * 16)); };
            if constexpr (RAW) {
                uint32_t top = 0u;
#pragma unroll
                for (int u = 0; u < DP / 8; ++u) {
                    const uint4 v = at(u);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                }
                uint32_t* const tops = reinterpret_cast<uint32_t*>(smem + L::TOPS) + lr;
                tops[part * kTileRows] = max(top & 0xffffu, top >> 16);
                named_bar_sync(row_bar, 32 * PARTS);
                top = tops[0];
#pragma unroll
                for (int k = 1; k < PARTS; ++k) top = max(top, tops[k * kTileRows]);
                // (E4M3's smallest step is 2^-9, f16's 2^-24: bf16's smallest number times 2^125 or 2^110 is one still)
                shift = NAT ? min(134 - (int)(top >> 7), 125) : min(131 - (int)(top >> 7), 110);
                f = exp2i(shift);
            }
            constexpr int NW = DP < 32 ? DP / 2 : 16;                 // words of two dims at a time
#pragma unroll 1
            for (int c = 0; c < DP / (2 * NW); ++c) {
                uint32_t w[NW];
#pragma unroll
                for (int u = 0; u < NW / 4; ++u) {
                    const uint4 v = at(NW / 4 * c + u);
                    w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
                }
#pragma unroll
                for (int k = 0; k < NW; ++k) {
                    // (0 times an infinity makes a NaN of it, for E4M3, which has none)
                    const float a = bf16_lo_to_f32(w[k]), b = bf16_hi_to_f32(w[k]);
                    w[k] = (NAT ? pack_f16x2(fmaf(a, f, a * 0.f), fmaf(b, f, b * 0.f)) : RAW ? pack_f16x2(a * f, b * f) : w[k]) ^ flip;
                }
                const uint32_t to = tmem + lanes_at + kColQ + (ic & 1) * (D / 2);
                if constexpr (NAT) {
                    uint32_t hi[NW / 2], lo[NW / 2];
#pragma unroll
                    for (int k = 0; k < NW / 2; ++k) {
                        const uint32_t a = f16x2_to_e4m3x2(w[2 * k]), b = f16x2_to_e4m3x2(w[2 * k + 1]);
                        hi[k] = a | b << 16;
                        lo[k] = f16x2_to_e4m3x2(sub_f16x2(w[2 * k], e4m3x2_to_f16x2((uint16_t)a))) |
                                f16x2_to_e4m3x2(sub_f16x2(w[2 * k + 1], e4m3x2_to_f16x2((uint16_t)b))) << 16;
                    }
                    tmem_st(to + part * (DP / 4) + NW / 2 * c, hi);
                    tmem_st(to + D / 4 + part * (DP / 4) + NW / 2 * c, lo);
                } else {
                    tmem_st(to + part * (DP / 2) + NW * c, w);
                }
            }
            named_bar_sync(row_bar, 32 * PARTS);                      // (the rows are read)
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQFull + (ic & 1)));
        return shift;
    };
    // Two: as operands, eight rows' 16-byte pieces side by side, and published later by the threads that
    // loaded them: lanes are 8 rows by 4 pieces.
    const uint32_t qdst = sbase + L::Q + h * L::QTILE + (uint32_t)(quarter * 512 + (lane & 7) * 16 + (lane >> 3) * 2048);
    auto load_q = [&](const Piece& x) {
        if (!busy(x)) return;
#pragma unroll 1
        for (int k = part; k < QB; k += PARTS) {                      // [8 rows of 32][4 pieces]
            const int r8 = k & 3, u = k & ~3, r = h * kTileRows + 32 * quarter + 8 * r8 + (lane & 7), token = r / p.G;
            const uint32_t to = qdst + r8 * 128 + u * 2048;
            if (token < x.tokens) cp_async_16(to, q_of(x, token, r - token * p.G) + 8 * (u + (lane >> 3)));
            else st_shared_v4(to, make_uint4(0u, 0u, 0u, 0u));
        }
        cp_async_commit();
    };
    auto publish_q = [&](const Piece& x) {
        cp_async_wait<0>();
        __syncwarp();
        if (flip && busy(x)) {
#pragma unroll 1
            for (int k = part; k < QB; k += PARTS) {
                const uint32_t to = qdst + (k & 3) * 128 + (k & ~3) * 2048;
                const uint4 v = ld_shared_v4(to);
                st_shared_v4(to, make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQFull + h));
    };
    Piece x{};
    bool ok = piece(0, x);
    if (ok) {
        if constexpr (SW == 2) load_q(x);
        else stage_q(x);
    }
    tc_fence_before();
    named_bar_sync(2, 32 * (W::SOFT + 1));
    tc_fence_after();
    tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::SLOT);
    const uint32_t lanes = tmem + lanes_at;
    const uint32_t ocol = kColO + (uint32_t)(h * kKeys);
    constexpr float kLift = RAW ? 7.f : 0.f;                          // (log2) on the probabilities
    int t0 = 0, ic = -1, next = 0;                                    // (the next tile of piece ic)
    if (ok) {
        if constexpr (SW == 2) publish_q(x);
        else shift = put_q(x, 0);
        ic = 0;
    }
    for (; ok; ++ic) {
        next = 0;
        const int n = x.n, rows = x.tokens * p.G;
        const bool live = busy(x), valid = tl < x.tokens;
        const int32_t* mrow = p.mask + (size_t)(x.qrow + (valid ? tl : 0)) * p.words;
        Piece y;
        ok = piece(ic + 1, y);
        if (!ok) break;
        if (SW == 1 && y.n > 0) stage_q(y);
        float m_used = -INFINITY, l = 0.f;
        int shift_next = 0;
        int ev = -1;
        // the row tile's warps without rows do not go through the keys: its first one arrives for them
        const int with_rows = PARTS * max(0, min(4, (rows - h * kTileRows + 31) / 32));
        const bool leads = warp % (4 * PARTS) == 0, runs = live || leads;
        const uint32_t arrivals = leads ? 4 * PARTS - with_rows + (with_rows > 0 ? 1 : 0) : 1;
        // The first tile by itself: the next piece's queries then follow outside the loop, which stays short
        // (with them in it, the instructions come too slowly: 64 ragged FP8 sequences of 4096 tokens, 32 nodes,
        // 189 us instead of 180; for the same reason a wait that does not end at once is a function, FP4 215 to 199).
        for (int lo = 0; ok && lo < n;) {
            int hi = SW == 1 && lo == 0 ? 1 : n, i = lo;
            bool wide = false;
#pragma unroll 1
            for (; runs && i < hi; ++i) {
                const int t = t0 + i, sb = SW == 2 ? h : t & 1;
                const uint32_t scol = kColS + (uint32_t)(sb * kKeys);
                // The first key as a node, of this thread's; FP8, whose columns are every other eight, of the tile's 128.
                const int first = (x.j0 + i) * kKeys + (NAT ? 0 : COLS * part) - x.start;
                // the visible keys of 32 columns are the bits of a word: the context's, then the row's mask
                uint32_t see[NC];
                const bool full = first + (NAT ? kKeys : COLS) <= 0;
                if (live && !full) {
                    auto word = [&](int node) { return valid ? seen_word(mrow, p.words, node, x.nodes) : 0u; };
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int at = part * NC + c;                     // of the tile's four: FP8: [slots' half][blocks' half]
                        see[c] = NAT ? __byte_perm(word(first + 64 * (at & 1)), word(first + 64 * (at & 1) + 32), at & 2 ? 0x7531 : 0x6420)
                                     : word(first + 32 * c);
                    }
                }
                ok = warp_wait(bar(kSFull + sb), SW == 2 ? (t & 1) : ((t >> 1) & 1));
                if (!ok) break;
                if (live) {
                    tc_fence_after();
                    float c1 = scale;
                    float drop = 1.f;                                     // what a change of V's power of two puts on O
                    if constexpr (RAW) {
                        const uint2 e = ld_shared_v2(sbase + L::PASSED + (NAT ? sb * L::PASS + kKeys * 4 : 8 * (t & 7)));
                        if ((int)e.y != ev) {
                            // V's power of two changes (or the piece begins), or the tile is a wide one, each time
                            if (e.y > 0xffu || ev == kOwnUnits) {
                                wide = true;
                                break;
                            }
                            drop = exp2i(ev - (int)e.y);
                            ev = (int)e.y;
                        }
                        c1 *= exp2i(max(min((int)e.x - 127 - shift, 127), -126));
                    }
                    c1 = fmaxf(c1, FLT_MIN);                              // (a hidden key's -inf stays -inf under a scale of 0)
                    const uint32_t mine = lanes + scol + COLS * part;
                    uint32_t sr[32];
                    // 32 of the thread's columns, hidden keys' -inf (a select: unread or stale columns may hold NaN)
                    auto scores = [&](int c) {
                        tmem_ld32(mine + 32 * c, sr);
                        uint4 sk[NAT ? 8 : 1];
                        if constexpr (NAT) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) sk[k] = ld_shared_v4(sbase + L::PASSED + sb * L::PASS + 4 * (COLS * part + 32 * c + 4 * k));
                        }
                        tmem_wait_ld();
                        if constexpr (NAT) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const uint64_t a = mul2((uint64_t)sr[k + 1] << 32 | sr[k], (uint64_t)sk[k / 4].y << 32 | sk[k / 4].x);
                                const uint64_t b = mul2((uint64_t)sr[k + 3] << 32 | sr[k + 2], (uint64_t)sk[k / 4].w << 32 | sk[k / 4].z);
                                sr[k] = (uint32_t)a;
                                sr[k + 1] = (uint32_t)(a >> 32);
                                sr[k + 2] = (uint32_t)b;
                                sr[k + 3] = (uint32_t)(b >> 32);
                            }
                        }
                    };
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        scores(c);
                        if (!full) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((see[c] >> k) & 1u)) sr[k] = 0xff800000u;
                            if (NC > 1) tmem_st32(mine + 32 * c, sr);
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], __uint_as_float(sr[k]), __uint_as_float(sr[k + 1]));
                    }
                    if (NC > 1 && !full) tmem_wait_st();
                    float mx = max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * c1;
                    // whether a row of the warps rises, or V's power of two
                    const bool rise = named_bar_or(row_bar, 32 * PARTS, mx > m_used + kRaise || drop != 1.f);
                    float alpha = 1.f;
                    if (rise) {
                        shared_row[part * kTileRows] = mx;
                        named_bar_sync(row_bar, 32 * PARTS);
#pragma unroll
                        for (int k = 0; k < PARTS; ++k) mx = fmaxf(mx, shared_row[k * kTileRows]);
                        if (mx > m_used + kRaise) {                       // (the first keys: from -inf)
                            alpha = fast_exp2(m_used - mx);
                            m_used = mx;
                        }
                        if (i > 0) {
                            // with S double-buffered, S(t) complete does not imply P V(t - 1) complete
                            if (SW == 1) {
                                ok = warp_wait(bar(kPVDone), (t - 1) & 1);
                                tc_fence_after();
                            }
                            const float on_o = alpha * drop;
#pragma unroll 1
                            for (int c = 0; c < DP / 16 && ok; ++c) {
                                uint32_t o[16];
                                tmem_ld(lanes + ocol + part * DP + 16 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * on_o);
                                tmem_st(lanes + ocol + part * DP + 16 * c, o);
                            }
                        }
                        named_bar_sync(row_bar, 32 * PARTS);                     // (the maxima are read)
                        if (!ok) {
                            ++i;
                            break;
                        }
                    }
                    // probabilities, rounded to the tensor cores' type (the sums take them unrounded: the
                    // roundings are of either sign and average out), over the first columns of this thread's part of S
                    const float m_sub = (m_used == -INFINITY ? 0.f : m_used) - kLift;
                    const uint64_t c2 = pair_of(c1, c1), nm2 = pair_of(-m_sub, -m_sub);
                    uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll (RAW ? 1 : 2)
                    for (int c = 0; c < NC; ++c) {
                        uint32_t pk[16];
                        if constexpr (NC > 1) scores(c);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const uint64_t y = fma2(pair_of(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), c2, nm2);
                            const float e0 = fast_exp2(pair_lo(y)), e1 = fast_exp2(pair_hi(y));
                            sum2[(k >> 1) & 1] = add2(sum2[(k >> 1) & 1], pair_of(e0, e1));
                            pk[k >> 1] = RAW ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
                        }
                        tmem_st16(mine + 16 * c, pk);
                    }
                    const uint64_t sum = add2(sum2[0], sum2[1]);
                    l = l * alpha + (pair_lo(sum) + pair_hi(sum));
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(bar(kPFull + sb), arrivals);
            }
            if constexpr (RAW) {
                if (wide) {
                    const WideRow r = wide_tile<D, T>(WideRow{m_used, l, ev, true}, sbase, tmem, t0 + i, i == 0, valid ? mrow : nullptr,
                                                      p.words, (x.j0 + i) * kKeys - x.start, x.nodes, shift, scale, kLift);
                    m_used = r.m;
                    l = r.l;
                    ev = r.ev;
                    ok = r.ok;
                    hi = ++i;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive_n(bar(kPFull + ((t0 + i - 1) & 1)), arrivals);
                }
            }
            next = ok ? hi : i;
            // (one row tile: the last piece's scores are taken, their Q is free)
            if (SW == 1 && ok && lo == 0 && y.n > 0) shift_next = put_q(y, ic + 1);
            lo = hi;
        }
        if (!ok) break;
        // (two: this piece's scores are taken, their Q is free)
        if (SW == 2 && y.n > 0) load_q(y);
        ok = warp_wait(bar(kODone + h), ic & 1);
        if (!ok) break;
        tc_fence_after();
        if (live) {
            // the row's sum, of its parts in their order
            shared_row[part * kTileRows] = l;
            named_bar_sync(row_bar, 32 * PARTS);
            l = shared_row[0];
#pragma unroll
            for (int k = 1; k < PARTS; ++k) l += shared_row[k * kTileRows];
            const bool whole = x.whole;
            const size_t piece = (size_t)(2 * blockIdx.x + (ic == 0 ? 0 : 1));
            const size_t orow = ((size_t)(x.qrow + tl) * p.Hq + (size_t)x.h * p.G + g) * D;
            // what is left on O: V's power of two, the probabilities' lift where the sums do not share it
            if (RAW && ev == kOwnUnits) ev = (int)ld_shared_u32(sbase + L::UNITS + 4 * (kTileRows * part + lr));
            const float back = RAW ? exp2i(ev - 127) : 1.f;
            const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : exp2i(-(int)kLift);
            constexpr int EC = DP < 32 ? DP : 32;
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0u;
#pragma unroll 1
            for (int c = 0; c < DP / EC; ++c) {
                uint32_t o[EC];
                const int col = part * DP + EC * c;
                tmem_ld(lanes + ocol + col, o);
                tmem_wait_ld();
                if (valid) {
#pragma unroll
                    for (int k = 0; k < EC; ++k) {
                        float y = __uint_as_float(o[k]) * inv;
                        if (RAW) y *= back;
                        o[k] = __float_as_uint(inv != 0.f ? y : 0.f);     // (no key that the row sees: O may be anything)
                    }
                    if (whole) {
                        uint16_t* dst = static_cast<uint16_t*>(p.out) + orow + col;
#pragma unroll
                        for (int v = 0; v < EC / 16; ++v) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * k]), __uint_as_float(o[16 * v + 2 * k + 1]));
                            if (wide) {
                                st_global_v8(dst + 16 * v, w);
                            } else {
                                reinterpret_cast<uint4*>(dst + 16 * v)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                reinterpret_cast<uint4*>(dst + 16 * v)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(p.part_o) + (piece * (D / 4) + col / 4) * p.slot_rows + row;
#pragma unroll
                        for (int v = 0; v < EC / 4; ++v)
                            dst[(size_t)v * p.slot_rows] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    }
                }
                __syncwarp();
            }
            if (valid && !whole && part == 0) p.part_ml[piece * p.slot_rows + row] = make_float2(m_used, l * exp2i(-(int)kLift));
            if (valid && *reinterpret_cast<volatile uint32_t*>(smem + L::ODD + 4 * (ic & 1)) != 0u) {
                // the rare values that are no finite numbers, of the tokens that the row sees, on what was stored
                const int32_t* trow = p.tables + (size_t)x.s * p.max_blocks;
                for (int tok = max(x.start, x.j0 * kKeys); tok < min(x.end(), (x.j0 + n) * kKeys); ++tok) {
                    const int node = tok - x.start;
                    if (!(((uint32_t)__ldg(mrow + node / 32) >> (node & 31)) & 1u)) continue;
                    const int32_t blk = __ldg(trow + tok / kBlockTokens);
                    if (blk < 0 || blk >= p.num_blocks) continue;
                    const char* rec = p.v_pool + ((size_t)blk * p.Hkv + x.h) * (size_t)REC;
#pragma unroll 1
                    for (int d = part * DP; d < (part + 1) * DP; ++d) {
                        const float y = value_at<D, T>(rec, tok % kBlockTokens, d);
                        if (fabsf(y) <= FLT_MAX) continue;
                        if (whole) {
                            __nv_bfloat16* at = static_cast<__nv_bfloat16*>(p.out) + orow + d;
                            *at = __float2bfloat16_rn(__bfloat162float(*at) + y);
                        } else {
                            p.part_o[((piece * (D / 4) + d / 4) * p.slot_rows + row) * 4 + d % 4] += y;
                        }
                    }
                }
            }
        }
        // O is read: the next piece's P V may start afresh
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kOFree));
        piece_done(ic);
        t0 += n;
        if (y.n == 0) break;
        x = y;
        if constexpr (SW == 2) publish_q(x);
        else shift = shift_next;
    }
    if (!ok) {
        if (lane == 0) raise_flag(p.err, PA_DEV_ERR_TIMEOUT);
        rows_leave<D, SW, PARTS, RAW>(p, reinterpret_cast<const Walk*>(smem + L::FIRST), ic, next, row, row_bar, shared_row + part * kTileRows);
    }
    // (no query copy may still be landing when the CTA ends)
    cp_async_wait<0>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W::MMA) {
        tc_fence_after();
        tmem_dealloc<512>(*reinterpret_cast<volatile uint32_t*>(smem + L::SLOT));
    }
}

template <int D, pa_dtype T, int SW>
cudaError_t launch(const TreeArgs& a, cudaStream_t stream) {
    constexpr int smem = Layout<D, T, SW>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<D, T, SW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(tree_sms(), kTreeCtas);
    const TParams p = tree_params(a, SW * kTileRows, ctas);
    e = tree_launch(tree_tc_kernel<D, T, SW>, dim3(ctas), Roles<T, SW>::THREADS, smem, stream, p);
    return e != cudaSuccess ? e : launch_merge<D, __nv_bfloat16>(p, stream);
}

template <int D>
cudaError_t launch_type(const TreeArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case PA_BF16:
            return tree_tile_rows((long long)a.num_q_heads / a.num_kv_heads * a.max_chunk) > kTileRows ? launch<D, PA_BF16, 2>(a, stream)
                                                                                                    : launch<D, PA_BF16, 1>(a, stream);
        case PA_FP8_E4M3: return launch<D, PA_FP8_E4M3, 1>(a, stream);
        case PA_FP4_E2M1: return launch<D, PA_FP4_E2M1, 1>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
    return a.head_dim == 64 ? launch_type<64>(a, stream) : launch_type<128>(a, stream);
}

}  // namespace pa
