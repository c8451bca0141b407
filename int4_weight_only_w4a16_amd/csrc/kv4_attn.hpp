// What the attention kernels of the 4-bit key/value cache share: a workgroup's rows and
// slots, the plan of a launch, LDS access.
#pragma once

#include <algorithm>

#include "kv4_device.hpp"
#include "lds.hpp"

namespace w4a16 {

// A launch: rows of a workgroup's tile of rows, tiles of rows, tiles of slots of a workgroup
// (a chunk), chunks.  Partial results of one (sequence, head, tile of rows, chunk): rows x (D
// sums), rows references, rows sums of p.
struct Plan {
    int rows, row_tiles, chunk, chunks;
};

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kNone = -3e38f;        // reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
// The activation type's largest number: m + 15 s may lie past it by the rounding of s, and an
// infinite high part would make the low part, and the row, NaN.
template <bool BF>
constexpr float kLargest = BF ? 3.3895314e38f : 65504.0f;

// What a workgroup works on: a tile of rows of one head of one sequence, and
// a range of its slots.
struct Work {
    int b, h, len, n, first;      // sequence, head, slots, new tokens, row of q of the first new token
    int start;                    // slot of the first new token
    int row0, rows;               // first row of the tile; rows of the sequence
    int t0, t1;                   // tiles of slots that any row of the tile sees
};

// Which part of the work a workgroup takes: a chunk of slots, a head's tile of rows (the tile-th, head
// group % kv_heads) of `groups`, a sequence.  The launches for trees have the chunks outermost: sequences
// differ in length, and chunks that only some have would, innermost, keep some XCDs (block index modulo 8)
// busier than others (12 trees over 900 to 12000 slots, four chunks:
// 143 us for the call; 106 with them outermost).
struct Place {
    int chunk, group, groups, batch;
};
template <bool TREE>
__device__ __forceinline__ Place place_of(const Plan &plan, int kv_heads) {
    const int groups = kv_heads * plan.row_tiles;
    if (TREE) return {(int)(blockIdx.x / groups), (int)(blockIdx.x % groups), groups, (int)blockIdx.y};
    return {(int)blockIdx.x, (int)blockIdx.y, groups, (int)blockIdx.z};
}
inline dim3 tree_grid(const Kv4AttnArgs &a, const Plan &p) {
    return dim3((unsigned)(a.c.kv_heads * p.row_tiles * p.chunks), (unsigned)a.c.batch);
}

__device__ __forceinline__ bool work_of(const Kv4AttnArgs &a, int b, int h, int row0, int rows_per, Work *w) {
    const int64_t first = a.cu[b], end = a.cu[b + 1], kv_len = max(a.kv_len[b], 0);
    const int64_t n64 = min(end, a.T) - first;
    if (first < 0 || n64 <= 0) return false;
    w->b = b;
    w->h = h;
    w->first = (int)first;
    // the limits cut off rows and slots; where a token sits does not depend on them
    w->n = (int)min(n64, (int64_t)a.max_q);
    w->start = (int)max(kv_len - (end - first), (int64_t)-0x3fffffff);
    const int64_t cap = (int64_t)a.c.table_stride * a.c.tiles_per_page * 32;
    w->len = (int)min(min(kv_len, (int64_t)a.max_kv), cap);
    const int G = a.q_heads / a.c.kv_heads;
    w->row0 = row0;
    w->rows = w->n * G;
    if (row0 >= w->rows) return false;
    const int last = min(row0 + rows_per, w->rows) - 1;
    // (in a tree a later token may lie less deep and see earlier slots)
    const int lo = row_lo(a.tree ? 0 : row0 / G, w->start, a.window);
    const int hi = row_hi(last / G, w->start, w->len, a.causal);
    w->t0 = lo >> 5;
    w->t1 = hi > lo ? (hi + 31) >> 5 : w->t0;
    return true;
}

// What drafted token i of a tree sees of the new tokens: bit j for token j, the earlier ones that it
// descends from and its own.  (Bits from i on that the word may hold mean nothing.)
__device__ __forceinline__ uint64_t kin_of(uint64_t word, int i) { return (word & ((1ull << i) - 1)) | 1ull << i; }

// Bit s: a row with the bounds [lo, hi) sees slot first + s of a tile's 32; `start` is the slot of the
// first new token, and hi at most 64 after it.
__device__ __forceinline__ uint32_t seen_bits(uint64_t kin, int lo, int hi, int start, int first) {
    const int from = min(max(lo - first, 0), 32), to = min(max(hi - first, from), 32);
    const int before = min(max(start - first, 0), 32), past = min(max(first - start, 0), 63);
    const uint32_t in_tree = (uint32_t)((1ull << before) - 1) | (uint32_t)((kin >> past) << before);
    return (uint32_t)((1ull << to) - (1ull << from)) & in_tree;
}

// Tiles of a workgroup that walks over one of about `want` equal parts of `tiles`, a whole number
// for each wave.  The page ids of a part sit in the 64 lanes of a wave, 62 of them wherever it
// begins; parts that this bounds stay equal (4000 slots of 64-slot pages, 192 rows, 32 sequences:
// 287 us in two halves, 453 as 124 tiles and one).
inline int chunk_of(const Kv4Cache &c, int tiles, int64_t want) {
    if (c.tiles_per_page < (1 << 20)) {
        const int64_t most = 62 * (int64_t)c.tiles_per_page / kWaves * kWaves;
        want = std::max(want, (tiles + most - 1) / most);
    }
    const int64_t chunk = ((tiles + want - 1) / want + kWaves - 1) / kWaves * kWaves;
    return (int)std::max<int64_t>(kWaves, chunk);
}

}  // namespace

// The kernel for many rows, the rows of its tiles and its plan (kv4_prefill_gfx950.hip).
int prefill_rows(int head_dim);
Plan prefill_plan(const Kv4AttnArgs &a);
hipError_t launch_kv4_prefill(const Kv4AttnArgs &a, const Plan &p, hipStream_t stream);

}  // namespace w4a16
