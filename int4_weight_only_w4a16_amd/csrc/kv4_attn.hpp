// What the attention kernels of the 4-bit key/value cache share: a workgroup's rows and
// slots, the plan of a launch, LDS access.
#pragma once

#include <algorithm>

#include "kv4_device.hpp"

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
    const int lo = row_lo(row0 / G, w->start, a.window);
    const int hi = row_hi(last / G, w->start, w->len, a.causal);
    w->t0 = lo >> 5;
    w->t1 = hi > lo ? (hi + 31) >> 5 : w->t0;
    return true;
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

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) void lds_void;
template <typename T>
__device__ __forceinline__ T lds_get(const lds_u8 *p) {
    return *reinterpret_cast<const __attribute__((address_space(3))) T *>(p);
}
template <typename T>
__device__ __forceinline__ void lds_put(lds_u8 *p, T v) {
    *reinterpret_cast<__attribute__((address_space(3))) T *>(p) = v;
}

// One KiB from `base + at` to LDS without passing through registers, lane l's 16 bytes to 16 l; what
// lies at or past base + bytes comes as zeros.
__device__ __forceinline__ void copy_kib(const uint8_t *base, uint32_t bytes, uint32_t at, lds_u8 *to, int lane) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, bytes), (lds_void *)to, 16, 16 * lane, at, 0, 0);
}

// A workgroup barrier for LDS alone: this wave's LDS operations are done, and loads from memory
// stay under way (__syncthreads waits for those too).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// s_waitcnt vmcnt(n): at most n of this wave's vector memory instructions are still under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

}  // namespace

// The kernel for many rows, the rows of its tiles and its plan (kv4_prefill_gfx950.hip).
int prefill_rows(int head_dim);
Plan prefill_plan(const Kv4AttnArgs &a);
hipError_t launch_kv4_prefill(const Kv4AttnArgs &a, const Plan &p, hipStream_t stream);

}  // namespace w4a16
