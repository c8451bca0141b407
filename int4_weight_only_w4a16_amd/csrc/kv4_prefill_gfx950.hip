// Softmax attention over the 4-bit key/value cache for many rows at a time
// (prompts and chunks of prompts).
//
// Rows are (new token, query head of the group) pairs.  A workgroup takes
// 256 rows (128 with 256 channels), 32 in each of its waves, and walks over
// the slots 64 at a time: two tiles of the cache are unpacked once into LDS,
// as the matrix operands of all waves, while the previous two are worked on.
//   x_t = sum_g s_g (q_g . (B + c_g)) + sum_g (m_g - B s_g) sum(q_g)
// the first products on the exact 16-bit numbers B + c (B = 64 or 128), the
// second sum a matrix product too: both factors in three bfloat16 parts of
// eight bits, the six products of parts that matter at 24 bits (its rounding
// is that of the fp32 sums).  So a weight takes one fma a group, and
//   p_t = exp2(scale log2(e) x_t - ref),  out = sum_t p_t v_t / sum_t p_t
// with v_t = m + s c unpacked into two parts of the activation type (high and
// low: 2^-17 or better of v_t) and p_t rounded to it for the second product.
// So values cost all waves one unpacking and the weights nothing a group, and
// only the p_t are rounded: with values of one part the result is off by
// sqrt(3) roundings of the output instead of sqrt(2) (measured 2.8e-3 instead
// of 2.4e-3 in bfloat16; the plain form's one rounding is 1.7e-3).  The
// matrix cores have the time for the low parts.
//
// Bound by the matrix cores and the vector ALUs, which one wave does not keep busy together: two
// prompts of 1500 and 2500 tokens over 12000 and 6000 slots, 40 heads on 8 (589 GFLOP of the
// formula's products, 920 with the low parts and the offset term) 1008 us, 584 TFLOP/s of the
// former.  A large product alone reaches 1280.  Fetching and unpacking, shared by the 8 waves, is
// about a third of it.
//
// The transposed products K Q^T and V^T P^T put a row of the softmax in one
// column: a lane's weights are the second product's operand as they stand,
// if the 32 slots of a tile are the first operand's rows in the order
// row(slot) = slot with bits 3 and 4 exchanged.

#include <algorithm>

#include "kv4_attn.hpp"

namespace w4a16 {
namespace {

// The weights stay below 2^(kLiftMany + kSlackMany).  fp16 has few numbers below 2^-14 and none below
// 2^-25, so there the reference lies below the maximum: a rounding is relative down to 2^-21 of
// the largest weight instead of 2^-14.
constexpr float kSlackMany = 8.0f;
template <bool BF>
constexpr float kLiftMany = BF ? 0.0f : 7.0f;
constexpr int kPairs = 6;              // products of parts

__device__ __forceinline__ int part_of_offset(int pair) { return (0x011002 >> (4 * (5 - pair))) & 15; }
__device__ __forceinline__ int part_of_sum(int pair) { return (0x010120 >> (4 * (5 - pair))) & 15; }

template <int D>
constexpr int kManyThreads = D <= 128 ? 512 : 256;

template <int D, int NG>
struct ManyShape {
    using T = Tile<D, NG>;
    static constexpr int kWaves = kManyThreads<D> / 64;
    static constexpr int kRows = 32 * kWaves;
    static constexpr int kTiles = D <= 128 ? 2 : 1;             // tiles of a stage
    static constexpr int kTerms = (kPairs * NG + 3 + 15) / 16;  // 16-deep products of the offset term
    // one stage: the tiles' key operands, value operands, offset operands, steps, NaN masks
    static constexpr int kKeys = 64 * D;                        // bytes of one tile's
    static constexpr int kValues = 128 * D;                     // high parts, then low parts
    static constexpr int kOffsets = 1024 * kTerms;
    static constexpr int kSteps = 128 * NG;
    static constexpr int kAtValues = kTiles * kKeys;
    static constexpr int kAtOffsets = kAtValues + kTiles * kValues;
    static constexpr int kAtSteps = kAtOffsets + kTiles * kOffsets;
    static constexpr int kAtBad = kAtSteps + kTiles * kSteps;
    static constexpr int kStage = kAtBad + 80;
    static_assert(4 + kTiles * NG * 4 <= 80, "NaN masks");
    // the packed tiles on their way: a ring of three stages' worth, a KiB a copy instruction
    static constexpr int kRawTile = (T::kBytes + 1023) / 1024 * 1024;
    static constexpr int kRing = 3;
    static constexpr int kCopies = (kTiles * kRawTile / 1024 + kWaves - 1) / kWaves;     // of a stage in each wave
    static constexpr int kAtRaw = 2 * kStage / 1024 * 1024 + 1024;
    static constexpr int kLds = kAtRaw + kRing * kTiles * kRawTile;
};

__device__ __forceinline__ int row_of_slot(int s) { return (s & 7) | (s & 8) << 1 | (s & 16) >> 1; }

// TREE: the new tokens are a tree of drafts, as in the kernel for few rows.
template <bool BF, int D, int NG, bool TREE>
__global__ void __launch_bounds__(kManyThreads<D>)
    __attribute__((amdgpu_waves_per_eu(D <= 128 ? 2 : 1, D <= 128 ? 2 : 1))) prefill_kernel(Kv4AttnArgs a, Plan plan) {
    using T = Tile<D, NG>;
    using Shape = ManyShape<D, NG>;
    constexpr int kTerms = Shape::kTerms, kWaves = Shape::kWaves, kTiles = Shape::kTiles, kRing = Shape::kRing;
    constexpr int kDeep = D / 16;                 // 16-channel products
    constexpr int kPer = kDeep / NG;              // of them per group
    constexpr int kOut = D / 32;                  // 32-channel blocks of the output
    // codes of a stage: kAll KiB of keys and as much of values, in each wave kWords of the four
    // words that a lane of one such KiB has
    constexpr int kAll = kTiles * (D / 64), kParts = kWaves / kAll, kWords = 4 / kParts;
    static_assert(kAll * kParts == kWaves && kWords * kParts == 4, "every wave has the same share");
    constexpr int kValGroups = T::kGroup == 32 && kWords == 4 ? 2 : 1;     // groups that they touch
    __shared__ __align__(16) uint8_t lds_raw[Shape::kLds];
    lds_u8 *const lds = (lds_u8 *)lds_raw;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int kvh = a.c.kv_heads, G = a.q_heads / kvh;
    const Place me = place_of<TREE>(plan, kvh);
    Work w;
    // later rows see more slots: the longest tiles of rows first
    const int row_tile = plan.row_tiles - 1 - me.group / kvh;
    if (!work_of(a, me.batch, me.group % kvh, row_tile * Shape::kRows, Shape::kRows, &w)) return;
    const int chunk0 = w.t0 + me.chunk * plan.chunk;
    const int chunk1 = min(chunk0 + plan.chunk, w.t1);
    if (me.chunk > 0 && chunk0 >= w.t1) return;

    // ---- this lane's column: a row of q, its channels as matrix operands, what it sees ----
    const int row = w.row0 + 32 * wave + col;
    const bool in_seq = row < w.rows;
    const int token = in_seq ? row / G : 0, head = w.h * G + (in_seq ? row - token * G : 0);
    uint64_t of_tree = 0;
    int depth = token;
    if constexpr (TREE) {
        of_tree = in_seq ? kin_of(a.tree[w.first + token], token) : 0;
        depth = __popcll(of_tree) - 1;
    }
    const int lo = in_seq ? row_lo(depth, w.start, a.window) : 0;
    const int hi = in_seq ? row_hi(token, w.start, w.len, a.causal) : 0;
    u4 q[kDeep], sums[kTerms];
    {
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + (int64_t)(w.first + token) * a.q_stride +
                              (int64_t)head * D + 8 * half;
        float qsum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) qsum[g] = 0.f;
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            q[j] = *reinterpret_cast<const u4 *>(src + 16 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) qsum[j / kPer] += lo_f32<BF>(q[j][e]) + hi_f32<BF>(q[j][e]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) qsum[g] += __shfl_xor(qsum[g], 32);
        // place k of the offset term's depth: pair k / NG of group k % NG
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[2] = {0.f, 0.f};
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {          // (both halves' places are compile-time)
                        const int k = 16 * t + 8 * hh + 2 * e + o;
                        if (k < kPairs * NG) {
                            const float p = bf16_part(qsum[k % NG], part_of_sum(k / NG));
                            if (half == hh) v[o] = p;
                        }
                    }
                sums[t][e] = pack2<true>(v[0], v[1]);
            }
    }
    // the slots that every row of the wave sees
    int all_lo = in_seq ? lo : 0, all_hi = in_seq ? hi : 0x7fffffff;
    if constexpr (TREE) all_hi = min(all_hi, w.start);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        all_lo = max(all_lo, __shfl_xor(all_lo, d));
        all_hi = min(all_hi, __shfl_xor(all_hi, d));
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    // ---- packed tiles into the ring ----
    // 64 page ids at a time sit in the lanes, so that no copy waits for one; (page, in) is where
    // the next tile to copy lies, `place` its address
    const int tpp = a.c.tiles_per_page;
    const int32_t *const table = a.c.table + (int64_t)w.b * a.c.table_stride;
    int window = chunk0 / tpp, page = window, in = chunk0 - window * tpp, next_tile = chunk0, ring_next = 0;
    auto load_ids = [&]() { return window + lane < a.c.table_stride ? table[window + lane] : -1; };
    int ids = load_ids();
    const uint8_t *place = nullptr;
    bool on_page = false;
    auto enter_page = [&]() {
        if (page - window >= 64) {
            window = page;
            ids = load_ids();
        }
        const int id = __builtin_amdgcn_readlane(ids, page - window);
        on_page = (unsigned)id < (unsigned)a.c.num_pages;
        place = a.c.pages + (((int64_t)(on_page ? id : 0) * kvh + w.h) * tpp + in) * T::kBytes;
    };
    enter_page();
    // copies the tiles of the next stage; bit t of the result: tile t is there
    auto copy = [&]() {
        uint32_t found = 0;
        const uint8_t *at[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            at[t] = place;
            found |= next_tile < chunk1 && on_page ? 1u << t : 0u;
            ++next_tile;
            place += T::kBytes;
            if (++in == tpp) {
                in = 0;
                ++page;
                if (next_tile < chunk1) enter_page();
            }
        }
#pragma unroll
        for (int i = 0; i < Shape::kCopies; ++i) {
            // (a wave without a copy of its own repeats the last one)
            constexpr int kPerTile = Shape::kRawTile / 1024;
            const int unit = min(wave + kWaves * i, kTiles * kPerTile - 1), t = unit / kPerTile, u = unit % kPerTile;
            const uint8_t *from = kTiles > 1 && t ? at[kTiles - 1] : at[0];
            copy_kib(from, found >> t & 1 ? T::kBytes : 0, 1024 * u,
                     lds + Shape::kAtRaw + (ring_next * kTiles + t) * Shape::kRawTile + 1024 * u, lane);
        }
        ring_next = ring_next + 1 == kRing ? 0 : ring_next + 1;
        return found;
    };

    // ---- unpacking: a stage's tiles from the ring, the same share in every wave ----
    const float c1 = a.scale * kLog2e;
    const CodeConsts cc = code_consts<BF>();
    const int r16 = lane & 15, b4 = lane >> 4;
    const int unit = wave / kParts, word0 = wave % kParts * kWords;
    const int unit_tile = unit / (D / 64), chunk64 = unit % (D / 64);
    auto unpack = [&](int tile, const lds_u8 *ring, lds_u8 *to) {
        const lds_u8 *const raw = ring + unit_tile * Shape::kRawTile;
        lds_u8 *const keys = to + unit_tile * Shape::kKeys;
        lds_u8 *const values = to + Shape::kAtValues + unit_tile * Shape::kValues;
        uint32_t kcodes[kWords], vcodes[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const lds_u8 *from = raw + 1024 * chunk64 + 16 * lane + 4 * word0;
            kcodes[k] = lds_get<uint32_t>(from + 4 * k);
            vcodes[k] = lds_get<uint32_t>(from + T::kCodes + 4 * k);
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const int word = 4 * chunk64 + word0 + k;
            const int row = row_of_slot(16 * (word / (D / 32)) + r16);
            const int j = 2 * (word % (D / 32)) + (b4 >> 1);
            lds_put(keys + 1024 * j + 16 * (32 * (b4 & 1) + row), based_codes<BF>(kcodes[k], cc));
        }
#pragma unroll
        for (int g = 0; g < kValGroups; ++g) {
            const int group = (64 * chunk64 + 16 * word0) / T::kGroup + g;
            const lds_u8 *const par = raw + 2 * T::kCodes + 128 * (NG + group) + 16 * b4;
            u4 p[2] = {lds_get<u4>(par), lds_get<u4>(par + 64)};
            const int left = w.len - 32 * (tile + unit_tile);
            if (left < 32) {                     // slots past the sequence's: their parameters mean nothing
                asm volatile("");
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (16 * (e >> 2) + 4 * b4 + (e & 3) >= left) p[e >> 2][e & 3] = 0u;
            }
            float st[8], off[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // NaN becomes a number here; the masks below bring it back
                st[e] = fmaxf(par_step<BF>(p[e >> 2][e & 3]), 0.f);
                off[e] = fmaxf(par_offset<BF>(p[e >> 2][e & 3]), -kLargest<BF>);
            }
#pragma unroll
            for (int k = g * kWords / kValGroups; k < (g + 1) * kWords / kValGroups; ++k) {
                uint32_t even = vcodes[k] & 0x0F0F0F0Fu, odd = (vcodes[k] >> 4) & 0x0F0F0F0Fu;
                asm("" : "+v"(even), "+v"(odd));
                u4 high, low;
#pragma unroll
                for (int e = 0; e < 4; ++e) {               // nibbles e and e + 4
                    const uint32_t src = e & 1 ? odd : even;
                    const float v0 = fminf(__builtin_fmaf(st[e], ubyte_f32(src, e >> 1), off[e]), kLargest<BF>);
                    const float v1 = fminf(__builtin_fmaf(st[4 + e], ubyte_f32(src, 2 + (e >> 1)), off[4 + e]), kLargest<BF>);
                    high[e] = pack2<BF>(v0, v1);
                    low[e] = pack2<BF>(v0 - lo_f32<BF>(high[e]), v1 - hi_f32<BF>(high[e]));
                }
                const int d = 64 * chunk64 + 16 * (word0 + k) + r16;
                lds_u8 *const to_value = values + 1024 * (2 * (d / 32) + (b4 >> 1)) + 16 * (32 * (b4 & 1) + d % 32);
                lds_put(to_value, high);
                lds_put(to_value + 64 * D, low);
            }
        }
    };
    auto parameters = [&](int tile, const lds_u8 *ring, lds_u8 *to) {
        const int t = kTiles > 1 ? lane >> 5 : 0, s = lane & 31;
        if (wave > 3) return;
        uint32_t kpar[NG];                       // wave 3: of the values
#pragma unroll
        for (int g = 0; g < NG; ++g)
            kpar[g] = lds_get<uint32_t>(ring + t * Shape::kRawTile + 2 * T::kCodes +
                                        128 * (g + (wave == 3 ? NG : 0)) + 4 * s);
        const bool lane_in = kTiles > 1 || lane < 32;        // (one tile: half a wave's slots)
        if (wave == 3) {
            // value groups with NaN: whether there are any, then a bit for each slot in use
            uint64_t any = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float st = par_step<BF>(kpar[g]);
                const uint64_t bad = __builtin_amdgcn_ballot_w64(lane_in && st != st && 32 * tile + lane < w.len);
                any |= bad;
                if (lane < kTiles) lds_put(to + Shape::kAtBad + 4 + 4 * (kTiles * g + lane), (uint32_t)(bad >> (32 * lane)));
            }
            if (lane == 0) lds_put(to + Shape::kAtBad, any ? 1u : 0u);
        } else if (wave == 2) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
                if (lane_in) lds_put(to + Shape::kAtSteps + t * Shape::kSteps + 4 * (32 * g + s), c1 * par_step<BF>(kpar[g]));
        } else if (wave < 2) {
            // offsets c1 (m - B s), half `wave` of each product's depth
            float off[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
                off[g] = c1 * __builtin_fmaf(-kCodeBase<BF>, par_step<BF>(kpar[g]), par_offset<BF>(kpar[g]));
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
                u4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f[2];
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        f[o] = 0.f;
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int k = 16 * term + 8 * hh + 2 * e + o;
                            if (wave != hh) continue;
                        if (k < kPairs * NG) f[o] = bf16_part(off[k % NG], part_of_offset(k / NG));
                        else if (k < kPairs * NG + 3) f[o] = 1.0f;       // the reference's parts
                        }
                    }
                    v[e] = pack2<true>(f[0], f[1]);
                }
                if (lane_in)
                    lds_put(to + Shape::kAtOffsets + t * Shape::kOffsets + 1024 * term + 16 * (32 * wave + row_of_slot(s)), v);
            }
        }
    };

    // ---- the softmax of a stage's 64 slots and its products ----
    // x = c1 q . k - ref comes out of the first products as it is: -ref, in three parts, has
    // places of its own in the offset term
    float ref = kNone, sum = 0.f, nans[NG];      // nans: NaN once the row saw one in that group, else 0
    f16v out[kOut];
    const f16v zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) nans[g] = 0.f;
#pragma unroll
    for (int o = 0; o < kOut; ++o) out[o] = zero;
    auto logits = [&](const lds_u8 *at, int t) {
        const lds_u8 *const keys = at + t * Shape::kKeys + 16 * lane;
        const lds_u8 *const steps = at + Shape::kAtSteps + t * Shape::kSteps + 16 * half;
        f16v x;
#pragma unroll
        for (int term = 0; term < kTerms; ++term)
            x = mfma32x32x16_t<true>(
                lds_get<u4>(at + Shape::kAtOffsets + t * Shape::kOffsets + 1024 * term + 16 * lane), sums[term],
                term ? x : zero);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f16v acc;
#pragma unroll
            for (int j = g * kPer; j < (g + 1) * kPer; ++j)
                acc = mfma32x32x16_t<BF>(lds_get<u4>(keys + 1024 * j), q[j], j % kPer ? acc : zero);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f4 st = lds_get<f4>(steps + 128 * g + 64 * (i & 1) + 32 * (i >> 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * i + e] = __builtin_fmaf(st[e], acc[4 * i + e], x[4 * i + e]);
            }
        }
        return x;            // register 4 i + e: slot 16 (i & 1) + 8 (i >> 1) + 4 half + e of the tile
    };
    auto move_reference = [&](float top, f16v (&x)[kTiles]) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const bool unset = ref == kNone;
        // (an infinite maximum stays out of the reference: its weight becomes infinite)
        float by = fminf(top, 3e38f) - kLiftMany<BF>;
        by = unset ? (top > -__builtin_inff() ? by : 0.f) : fmaxf(by, 0.f);
        const float f = unset ? 1.f : __builtin_amdgcn_exp2f(-by);
        ref = unset ? (top > -__builtin_inff() ? by : kNone) : ref + by;
        sum *= f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) x[t][i] -= by;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            constexpr int kFirst = kPairs * NG;
            const int k = kFirst + part, t = k / 16, e = k % 8 / 2;
            const uint32_t bits = pack2<true>(bf16_part(ref == kNone ? 0.f : -ref, part), 0.f);
            const uint32_t both = k % 2 ? (sums[t][e] & 0xFFFFu) | bits << 16 : (sums[t][e] & 0xFFFF0000u) | bits;
            if (half == k % 16 / 8) sums[t][e] = both;
        }
#pragma unroll
        for (int o = 0; o < kOut; ++o) out[o] *= f;
    };
    auto products = [&](const lds_u8 *at, int t, f16v &x) {
        const lds_u8 *const values = at + Shape::kAtValues + t * Shape::kValues + 16 * lane;
        u4 pw[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(x[i]);
            sum += x[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            pw[i >> 2][i & 3] = pack2<BF>(x[8 * (i >> 2) + (i & 3)], x[8 * (i >> 2) + 4 + (i & 3)]);
#pragma unroll
        for (int o = 0; o < kOut; ++o)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int part = 0; part < 2; ++part)
                    out[o] = mfma32x32x16_t<BF>(lds_get<u4>(values + 64 * D * part + 1024 * (2 * o + s)), pw[s], out[o]);
    };

    // ---- main loop: unpack the next stage while this one is worked on, the one after it on its way ----
    uint32_t found = copy(), found1 = copy(), found2 = 0;
    wait_loads<Shape::kCopies>();
    lds_barrier();
    auto raw_of = [&](int slot) { return lds + Shape::kAtRaw + slot * kTiles * Shape::kRawTile; };
    unpack(chunk0, raw_of(0), lds);
    parameters(chunk0, raw_of(0), lds);
    found2 = copy();
    wait_loads<Shape::kCopies>();
    lds_barrier();
    int stage = 0, ring_slot = 1;                // of the stage to unpack
    for (int tile = chunk0; tile < chunk1; tile += kTiles) {
        const lds_u8 *const at = lds + stage * Shape::kStage;
        stage ^= 1;
        lds_u8 *const to = lds + stage * Shape::kStage;
        const lds_u8 *const ring = raw_of(ring_slot);
        f16v x[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) x[t] = logits(at, t);
        // (pinned: else the last steps of x are taken past the branches below, and all their operands live on)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) asm volatile("" : "+v"(x[t]));
        unpack(tile + kTiles, ring, to);
        if (found != (1u << kTiles) - 1 || 32 * tile < all_lo || 32 * (tile + kTiles) > all_hi) {
            // (opaque bounds: the differences with them are not kept in registers from stage to stage)
            int from = lo - 32 * tile - 4 * half, to_slot = hi - 32 * tile - 4 * half;
            if constexpr (!TREE) asm volatile("" : "+v"(from), "+v"(to_slot));
            uint64_t kin = of_tree;
            int first_seen = lo, past_seen = hi;
            if constexpr (TREE && D == 256) {
                // what a row sees is made again for these few stages (opaque: it is not kept in registers, which are
                // short here: 176 bytes of a lane's in scratch, 152 so; with 128 channels, where they are not, it
                // costs 143 -> 163 us for 64 drafts over 65000 slots; with 256 it costs 310 -> 325 us for
                // 64 drafts over 30000 slots, groups of 32, and is for the scratch memory that a lane keeps)
                int again = lane;
                asm volatile("" : "+v"(again));
                again = w.row0 + 32 * wave + (again & 31);
                const int mine = again < w.rows ? again / G : 0;
                kin = again < w.rows ? kin_of(a.tree[w.first + mine], mine) : 0;
                first_seen = again < w.rows ? row_lo(__popcll(kin) - 1, w.start, a.window) : 0;
                past_seen = again < w.rows ? row_hi(mine, w.start, w.len, a.causal) : 0;
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if constexpr (TREE) {            // (selects: there are no branches for a lane's slots here)
                    const uint32_t there = found >> t & 1 ? ~0u : 0u;
                    const uint32_t bits =
                        (seen_bits(kin, first_seen, past_seen, w.start, 32 * (tile + t)) & there) >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[t][i] = bits >> (16 * ((i >> 2) & 1) + 8 * (i >> 3) + (i & 3)) & 1 ? x[t][i] : -__builtin_inff();
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int slot = 32 * t + 16 * ((i >> 2) & 1) + 8 * (i >> 3) + (i & 3);
                    if (!((found >> t & 1) & (slot >= from) & (slot < to_slot))) x[t][i] = -__builtin_inff();
                }
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, x[t][i]);
        if (__builtin_amdgcn_ballot_w64(top > kLiftMany<BF> + kSlackMany || (ref == kNone && top > -__builtin_inff())))
            move_reference(top, x);
        // a NaN that a row sees makes its group NaN
        if (__builtin_amdgcn_readfirstlane(lds_get<uint32_t>(at + Shape::kAtBad))) {
            asm volatile("");
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const uint32_t bad = lds_get<uint32_t>(at + Shape::kAtBad + 4 + 4 * (kTiles * g + t));
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int s = 16 * ((i >> 2) & 1) + 8 * (i >> 3) + 4 * half + (i & 3);
                        if ((bad >> s & 1) && x[t][i] != -__builtin_inff()) nans[g] = __builtin_nanf("");
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) products(at, t, x[t]);
        parameters(tile + kTiles, ring, to);
        found = found1;
        found1 = found2;
        found2 = copy();                         // over the tiles that were unpacked a stage ago
        ring_slot = ring_slot + 1 == kRing ? 0 : ring_slot + 1;
        wait_loads<Shape::kCopies>();            // this wave's copies of the stage after the next are there
        lds_barrier();
    }
    wait_loads<0>();

    // ---- the rows' results: register 4 i + e of block o holds channel 32 o + 8 i + 4 half + e ----
    const bool whole = w.t1 - w.t0 <= plan.chunk;
    float *part = static_cast<float *>(a.workspace) +
                  (((int64_t)w.b * me.groups + row_tile * kvh + w.h) * plan.chunks + me.chunk) * Shape::kRows * (D + 2);
    sum += __shfl_xor(sum, 32);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float nan = nans[g] + __shfl_xor(nans[g], 32);
#pragma unroll
        for (int o = g * kOut / NG; o < (g + 1) * kOut / NG; ++o)
#pragma unroll
            for (int i = 0; i < 16; ++i) out[o][i] += nan;
    }
    if (!in_seq) return;
    if (whole) {
        const int64_t at_q = w.first + token;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        uint16_t *to = static_cast<uint16_t *>(a.out) + at_q * a.out_stride + (int64_t)head * D + 4 * half;
#pragma unroll
        for (int o = 0; o < kOut; ++o)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<u2 *>(to + 32 * o + 8 * j) = pack4<BF>(
                    out[o][4 * j] * inv, out[o][4 * j + 1] * inv, out[o][4 * j + 2] * inv, out[o][4 * j + 3] * inv);
        if (a.lse && half == 0)
            a.lse[at_q * a.q_heads + head] =
                sum == 0.f ? -__builtin_inff() : (ref + __log2f(sum)) * (1.0f / kLog2e);
    } else {
        const int tile_row = 32 * wave + col;
#pragma unroll
        for (int o = 0; o < kOut; ++o)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f4 *>(part + (int64_t)tile_row * D + 32 * o + 8 * j + 4 * half) =
                    f4{out[o][4 * j], out[o][4 * j + 1], out[o][4 * j + 2], out[o][4 * j + 3]};
        if (half == 0) {
            part[Shape::kRows * D + tile_row] = ref;
            part[Shape::kRows * D + Shape::kRows + tile_row] = sum;
        }
    }
}

template <typename F>
hipError_t by_shape(const Kv4Cache &c, F f) {
    auto typed = [&](auto d, auto ng) {
        return c.bf16 ? f(std::true_type{}, d, ng) : f(std::false_type{}, d, ng);
    };
    return kv4_dispatch(c.head_dim, c.groups, typed);
}

}  // namespace

int prefill_rows(int head_dim) { return (head_dim <= 128 ? kManyThreads<128> : kManyThreads<256>) / 2; }

Plan prefill_plan(const Kv4AttnArgs &a) {
    Plan p;
    const int rows = a.q_heads / a.c.kv_heads * a.max_q;
    p.rows = prefill_rows(a.c.head_dim);
    p.row_tiles = (rows + p.rows - 1) / p.rows;
    int tiles = (a.max_kv + 31) / 32;
    if (a.window > 0) tiles = std::min(tiles, (a.window + std::min(a.max_q, p.rows)) / 32 + 2);
    // Split the slots where the tiles of rows alone leave some of the chip's 256 CUs without work (a
    // workgroup fills one): the number of parts with the least time, in us, of a model fitted to
    // 256 to 3200 rows over 2000 to 20000 slots.  A tile of slots is 1.5, a workgroup's start and
    // end 10, a part's partial results and their join 0.15.  (4 sequences of 2000 slots, 1600 rows:
    // 110 in one part, 203 in two; one of 20000: 964 in one, 281 in 4, 275 in 9, 300 in 18; 4800
    // rows of it: 967 in one, 674 in three.)
    const int64_t groups = (int64_t)a.c.batch * a.c.kv_heads * p.row_tiles;
    int64_t want = 1;
    if (groups < 512) {
        double least = 0;
        for (int64_t c = 1; c <= std::min<int64_t>(64, std::max(1, (tiles + 15) / 16)); ++c) {
            const int64_t rounds = (groups * c + 255) / 256, part = (tiles + c - 1) / c;
            const double time = (double)rounds * (1.5 * (double)part + 10) + (c > 1 ? 5 + 0.15 * (double)(groups * c) : 0);
            if (c == 1 || time < least) {
                least = time;
                want = c;
            }
        }
    }
    p.chunk = std::max<int>(16, (int)((tiles + want - 1) / want + 1) / 2 * 2);
    p.chunks = std::max(1, (tiles + p.chunk - 1) / p.chunk);
    return p;
}

hipError_t launch_kv4_prefill(const Kv4AttnArgs &a, const Plan &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.chunks, (unsigned)(a.c.kv_heads * p.row_tiles), (unsigned)a.c.batch);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        if (a.tree)
            prefill_kernel<bf(), d(), ng(), true><<<tree_grid(a, p), kManyThreads<d()>, 0, stream>>>(a, p);
        else
            prefill_kernel<bf(), d(), ng(), false><<<grid, kManyThreads<d()>, 0, stream>>>(a, p);
        return hipGetLastError();
    });
}

}  // namespace w4a16
