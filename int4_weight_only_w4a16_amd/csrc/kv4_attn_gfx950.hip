// Softmax attention over the 4-bit key/value cache.
//
// Rows are (new token, query head of the group) pairs; for row q and slot t
//   x_t = q . k_t,  k_t = m + s c per group of channels, B = 64 or 128
//       = sum_g s_g (q_g . (B + c_g) - B sum(q_g)) + m_g sum(q_g)
//   p_t = exp2(scale log2(e) x_t - ref),  out = sum_t p_t v_t / sum_t p_t,
//   sum_t p_t v_t = sum_t P_t (B + c_t) - (B + 8) sum_t P_t + sum_t p_t (m_t + 8 s_t),
//   P_t = p_t s_t rounded to the activation type.
// The codes go into the matrix instructions as the exact 16-bit numbers
// B + c; steps and offsets act on the fp32 sums.  The sum of the P_t comes
// from one more matrix product with ones, of the same rounded P_t, so that
// B + 8 comes off exactly and only P_t (c_t - 8) feels their rounding.
// A slot that a row does not see has p_t = 0 and adds nothing, whatever is
// stored there: its product with a step is the one in which 0 x anything is 0,
// and m + 8 s is held between the type's ends (a group with a NaN has it in
// both parameters, so that a slot with weight still gives NaN).
// Bound by memory while the rows are few, then by the vector ALUs (unpacking and weights): one
// token, 40 heads on 8, 131071 slots 30 us (4.7 TB/s of 5.2) and 4.6 for the join of chunks; 32
// sequences of 1000 to 24000 slots in groups of 32 119 us with a join of 5.6 (a call among others;
// the kernel by itself between pauses 125); 64 rows instead of 4 over 32 sequences of 4000 slots
// 104 us instead of 36.  A wave's tile comes while the one before is
// worked on; a third under way is slower (LDS for fewer waves: 9.1 -> 9.7 us at 2000 slots).
// ref is a running reference per row, moved only when a tile's maximum
// passes it by more than kSlack, and lies `lift` below the maximum: p_t stays
// below 2^(lift + kSlack).  fp16 has few numbers below 2^-14 and none below
// 2^-25, so there the weights start high: lift is 13, which rounds a P_t by at
// most 2^-38 of the largest weight, and less for rows that have met a step of
// 2 or more, so that P_t stays below 2^16.  (With 0 always, small values behind
// a dominant logit lost their weights: 5000 slots of 0.02, 12.5 below it, came
// out 0.29 % off, now 0.022 %, the output's rounding.)  bfloat16 has fp32's
// range: 0.

#include <algorithm>

#include "kv4_attn.hpp"

namespace w4a16 {
namespace {

constexpr float kSlack = 2.0f;
constexpr float kLift = 13.0f;         // the most

// a * b with 0 * anything = 0.
__device__ __forceinline__ float mul_legacy(float a, float b) {
    float r;
    asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// The larger of the low halves, and of the high halves, as whole numbers.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

// The largest of all lanes, in a scalar register.
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
#define W4A16_MAX_ROR(N) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true))
    W4A16_MAX_ROR(8);
    W4A16_MAX_ROR(4);
    W4A16_MAX_ROR(2);
    W4A16_MAX_ROR(1);
#undef W4A16_MAX_ROR
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

// v held to [-most, most]; a NaN becomes -most.
__device__ __forceinline__ float finite(float v, float most) { return __builtin_amdgcn_fmed3f(v, -most, most); }

// Chunks.  A few sequences: two workgroups for each CU, all of them at work at once, since a
// workgroup's start and end cost about as much as eight tiles (one sequence of 131071 slots, 8
// heads: 36.6 us with 512 workgroups, 39 with 1024, 43.6 with 2048).  More sequences may differ
// in length, and smaller chunks even that out (32 sequences of 1000 to 24000 slots: 136 us with
// 512, 123 with 1024 to 3072; of 4000 slots each: 36 with 1024, 39 with 1536, 49 with 4096).
constexpr int kFewSlots = 512, kManySlots = 1024, kFewSequences = 4;

// Rows above which the kernel for many rows runs, which keeps the matrix cores busier but works
// on 256 rows however few there are.  Here and there, 8 heads of 128 channels, bfloat16, us:
//   rows                            64           128          192          256          384
//   1 sequence of 100000 slots   65 and 176   138 and 183  177 and 189  233 and 201  325 and 339
//   8 of 4000                    43 and  76    63 and  88   83 and  97  105 and 107  152 and 167
//   32 of 4000                  104 and 239   196 and 268  288 and 296  378 and 325  562 and 420
// With 64 channels both meet near there too: at 192 rows 135 and 133, 68 and 70, 232 and 160; at
// 128 rows 107 and 131, 52 and 63, 160 and 159.  With 256 the kernel for many rows gains less (its
// tiles have 128 rows): at 192 rows 418 and 636, 150 and 238, 562 and 806; at 256 rows 551 and 638,
// 195 and 243, 743 and 808.
constexpr int kFewRows = 192;
int rows_of(const Kv4AttnArgs &a) { return a.q_heads / a.c.kv_heads * a.max_q; }

// 32 rows a wave read the cache half as often as 16, at two waves a SIMD instead of three (32
// rows, 32 sequences of 16000 slots: 184 us, 221 with 16; 8 of 4000: 33 and 31; 256 channels:
// 32 would not fit the registers)
int tile_rows(const Kv4AttnArgs &a) {
    if (rows_of(a) > kFewRows) return prefill_rows(a.c.head_dim);
    return rows_of(a) > 16 && a.c.head_dim <= 128 ? 32 : 16;
}

Plan plan_of(const Kv4AttnArgs &a) {
    const int rows = rows_of(a);
    if (rows > kFewRows) return prefill_plan(a);
    Plan p;
    p.rows = tile_rows(a);
    p.row_tiles = (rows + p.rows - 1) / p.rows;
    int tiles = (a.max_kv + 31) / 32;
    if (a.window > 0) tiles = std::min(tiles, (a.window + a.max_q) / 32 + 2);
    const int64_t groups = (int64_t)a.c.batch * a.c.kv_heads * p.row_tiles;
    // few slots: one chunk, and no join (one sequence of 256 slots: 8.6 -> 6.3 us, of 700: 8.7
    // with six chunks, 10.3 with one; 16 sequences of 1000: 15.0 -> 12.5 us)
    const int64_t want = tiles <= (groups >= 128 ? 32 : 16) ? 1 : std::max<int64_t>(
        1, (a.c.batch <= kFewSequences ? kFewSlots : kManySlots) / groups);
    p.chunk = chunk_of(a.c, tiles, want);
    p.chunks = std::max(1, (tiles + p.chunk - 1) / p.chunk);
    return p;
}

// One tile copied to LDS without passing through registers (lane l's 16 bytes of an
// instruction land at 16 l): the codes 1 KiB an instruction, the parameters 256 bytes, or
// 1 KiB where there are that many.  `bytes` 0 reads nothing and writes zeros.
template <int D, int NG>
struct TileCopy {
    using T = Tile<D, NG>;
    static constexpr bool kWidePar = NG % 4 == 0;
    static constexpr int kParLoads = kWidePar ? NG / 4 : NG;
    static constexpr int kLoads = D / 32 + kParLoads;       // instructions of a tile
    static __device__ __forceinline__ void issue(const uint8_t *tile, uint32_t bytes, lds_u8 *to, int lane) {
        const auto rsrc = make_rsrc(tile, bytes);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + 1024 * j), 16, 16 * lane, 1024 * j, 0, 0);
        constexpr int kAt = 2 * T::kCodes;
#pragma unroll
        for (int j = 0; j < kParLoads; ++j) {
            if constexpr (kWidePar)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + kAt + 1024 * j), 16, 16 * lane,
                                                         kAt + 1024 * j, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + kAt + 256 * j), 4, 4 * lane,
                                                         kAt + 256 * j, 0, 0);
        }
    }
};

// Up to 32 rows of one head against a chunk of slots.  Each wave takes every fourth tile of the
// chunk, on its own until the end.  Tiles go through a ring of kRing in LDS that is the wave's
// own: kRing - 1 are under way while one is worked on, and no barrier is needed.
template <int D, int NG, int NT>
struct AttendShape {
    using T = Tile<D, NG>;
    static constexpr int kRing = 2;
    static constexpr int kRows = 16 * NT;
    static constexpr int kOutRow = 4 * (D + 4);                            // bytes
    static constexpr int kTiles = kWaves * kRing * T::kBytes;
    static constexpr int kOuts = kWaves * kRows * kOutRow;                 // the waves' sums, at the end
    static constexpr int kStats = kTiles > kOuts ? kTiles : kOuts;         // references and sums of p
    static constexpr int kLds = kStats + 2 * kWaves * kRows * 4;
};

// TREE: the new tokens are a tree of drafts (up to 64): a row sees the slots before them and those
// that its token's word names.
template <bool BF, int D, int NG, int NT, bool TREE>
__global__ void __launch_bounds__(kThreads)
    __attribute__((amdgpu_waves_per_eu(NT * D <= 128 ? 3 : 2, NT * D <= 128 ? 3 : 2))) attend_kernel(Kv4AttnArgs a, Plan plan) {
    using T = Tile<D, NG>;
    using Shape = AttendShape<D, NG, NT>;
    using Copy = TileCopy<D, NG>;
    constexpr int kSteps = D / 32;            // 32-channel products of a slot
    constexpr int kPer = kSteps / NG;         // of them per group
    constexpr int kRows = Shape::kRows, kRing = Shape::kRing;
    constexpr int kOut = D / 16;              // 16-channel blocks of the output
    constexpr int kBlocks = kOut / NG;        // of them per group
    // Offsets of the values: with one group 24 operations in every lane, with more a matrix
    // product whose rows are the groups (about 36, whatever the number of groups).
    constexpr bool kMidRows = NG > 1;
    constexpr int kShare = NG > 1 ? NG / 2 : 1;       // of a tile's 32 NG value parameters, a lane's share
    __shared__ __align__(16) uint8_t lds_raw[Shape::kLds];
    lds_u8 *const lds = (lds_u8 *)lds_raw;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, b4 = lane >> 4;
    // The page ids of the chunk, one in each lane (the host keeps a chunk within 64 pages), so
    // that no copy waits for a page id.  Without a window a chunk's place does not depend on the
    // sequence's lengths, and the ids are loaded beside them.
    const int tpp = a.c.tiles_per_page, kvh = a.c.kv_heads;
    const Place me = place_of<TREE>(plan, kvh);
    auto load_ids = [&](int tile) {
        const int at = tile / tpp + lane;
        return at < a.c.table_stride ? a.c.table[(int64_t)me.batch * a.c.table_stride + at] : -1;
    };
    int ids = load_ids(me.chunk * plan.chunk);
    Work w;
    if (!work_of(a, me.batch, me.group % kvh, (me.group / kvh) * kRows, kRows, &w)) return;
    const int chunk0 = w.t0 + me.chunk * plan.chunk;
    const int chunk1 = min(chunk0 + plan.chunk, w.t1);
    if (me.chunk > 0 && chunk0 >= w.t1) return;
    const int G = a.q_heads / kvh;

    const int page0 = chunk0 / tpp;
    if (w.t0 > 0) ids = load_ids(chunk0);
    // (page, in): where the next copy's tile lies
    int next = chunk0 + wave, page = 0, in = chunk0 - page0 * tpp + wave, slot_next = 0;
    uint32_t there = 0;                       // bit s: the tile in ring slot s exists
    auto issue = [&]() {
        while (in >= tpp) {
            in -= tpp;
            ++page;
        }
        const int id = next < chunk1 ? __builtin_amdgcn_readlane(ids, page) : -1;
        const bool ok = (unsigned)id < (unsigned)a.c.num_pages;
        const uint8_t *p = a.c.pages + (((int64_t)(ok ? id : 0) * kvh + w.h) * tpp + in) * T::kBytes;
        Copy::issue(p, ok ? T::kBytes : 0, lds + (wave * kRing + slot_next) * T::kBytes, lane);
        there = (there & ~(1u << slot_next)) | ((ok ? 1u : 0u) << slot_next);
        slot_next = slot_next + 1 == kRing ? 0 : slot_next + 1;
        next += kWaves;
        in += kWaves;
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue();

    // this lane's columns: NT rows of q, their channels as matrix operands, and what they see
    u4 q[NT][kSteps], qparts[NT];
    float qsum[NT][NG];
    f4 init[NT][NG];                          // -B sum(q_g)
    int lo[NT], hi[NT];
    uint64_t kin[TREE ? NT : 1];
    int all_lo = 0, all_hi = TREE ? w.start : 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = w.row0 + 16 * t + r;
        const bool in_seq = row < w.rows;
        const int i = in_seq ? row / G : 0;
        int depth = i;
        if constexpr (TREE) {
            kin[t] = in_seq ? kin_of(a.tree[w.first + i], i) : 0;
            depth = __popcll(kin[t]) - 1;
        }
        lo[t] = in_seq ? row_lo(depth, w.start, a.window) : 0;
        hi[t] = in_seq ? row_hi(i, w.start, w.len, a.causal) : 0;
        if (in_seq) {
            all_lo = max(all_lo, lo[t]);
            all_hi = min(all_hi, hi[t]);
        }
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + (int64_t)(w.first + i) * a.q_stride +
                              (int64_t)(w.h * G + (in_seq ? row - i * G : 0)) * D + 8 * b4;
#pragma unroll
        for (int g = 0; g < NG; ++g) qsum[t][g] = 0.f;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            q[t][j] = *reinterpret_cast<const u4 *>(src + 32 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) qsum[t][j / kPer] += lo_f32<BF>(q[t][j][e]) + hi_f32<BF>(q[t][j][e]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            qsum[t][g] += __shfl_xor(qsum[t][g], 16);
            qsum[t][g] += __shfl_xor(qsum[t][g], 32);
            const float z = -kCodeBase<BF> * qsum[t][g];
            init[t][g] = f4{z, z, z, z};
        }
        // bfloat16: sum_g m_g sum(q_g) is one matrix product over 8 groups x 4 parts, the sums of q
        // in three parts of eight bits each (the m_g are exact)
        if constexpr (BF) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float z0 = 2 * e < NG ? qsum[t][2 * e < NG ? 2 * e : 0] : 0.f;
                const float z1 = 2 * e + 1 < NG ? qsum[t][2 * e + 1 < NG ? 2 * e + 1 : 0] : 0.f;
                qparts[t][e] = b4 < 3 ? pack2<BF>(bf16_part(z0, b4), bf16_part(z1, b4)) : 0u;
            }
        }
    }
    // the slots that every row sees, over the 16 columns
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
        all_lo = max(all_lo, __shfl_xor(all_lo, d));
        all_hi = min(all_hi, __shfl_xor(all_hi, d));
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    const float c1 = a.scale * kLog2e;
    const CodeConsts cc = code_consts<BF>();
    const uint32_t one16 = BF ? 0x3F803F80u : 0x3C003C00u;
    const u4 ones = {one16, one16, one16, one16};
    float ref[NT], sum[NT], lift[NT];
    uint32_t step_limit = 0x3FFF;        // fp16: the largest step, as bits, below 2^(14 - lift) of every row
    f4 out[NT][kOut], psum[NT][NG], mids[NT];      // mids: sum_t p_t (m_t + 8 s_t)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        ref[t] = kNone;
        sum[t] = 0.f;
        lift[t] = BF ? 0.f : kLift;
        mids[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < NG; ++g) psum[t][g] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int o = 0; o < kOut; ++o) out[t][o] = f4{0.f, 0.f, 0.f, 0.f};
    }

    // (of a tile's 32 slots this lane's eight are 16 (e / 4) + 4 b4 + e % 4)
    auto tree_bits = [&](int t, int tile) {
        return seen_bits(kin[TREE ? t : 0], lo[t], hi[t], w.start, 32 * tile) >> (4 * b4);
    };
    auto step = [&](int tile, const lds_u8 *at) {
        // whether some row does not see some of the tile's slots; the same in every lane
        const bool masked = 32 * tile < all_lo || 32 * tile + 32 > all_hi;
        const lds_u8 *params = at + 2 * T::kCodes + 16 * b4;
        // fp16: the largest step of the values, as bits, of the tile's parameters that fall to this lane
        uint32_t steps = 0;
        if constexpr (!BF) {
            const lds_u8 *all = at + 2 * T::kCodes + 128 * NG + 4 * kShare * (NG > 1 ? lane : lane & 31);
#pragma unroll
            for (int i = 0; i < kShare; ++i) steps = max_halves(steps, lds_get<uint32_t>(all + 4 * i));
            steps &= 0xFFFFu;
        }
        float x[NT][8];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            u4 kc[kSteps];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                if constexpr (D == 64) {
                    const u4 words = lds_get<u4>(at + 16 * lane);
                    kc[j] = based_codes<BF>(words[sub * kSteps + j], cc);
                } else if (j % 4 == 0) {
                    const u4 words = lds_get<u4>(at + 1024 * ((sub * kSteps + j) / 4) + 16 * lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kc[j + i] = based_codes<BF>(words[i], cc);
                }
            }
            if constexpr (BF) {
                u4 m = {0u, 0u, 0u, 0u};         // offsets of the slot that is this lane's row
                const lds_u8 *mine = at + 2 * T::kCodes + 64 * sub + 4 * r;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t p = lds_get<uint32_t>(mine + 128 * g);
                    m[g / 2] = g % 2 ? __builtin_amdgcn_perm(p, m[g / 2], 0x07060100u) : p >> 16;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const f4 z = mfma16x16x32_t<BF>(m, qparts[t], f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[t][4 * sub + e] = z[e];
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const u4 kp = lds_get<u4>(params + 128 * g + 64 * sub);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f4 acc = init[t][g];
#pragma unroll
                    for (int j = g * kPer; j < (g + 1) * kPer; ++j) acc = mfma16x16x32_t<BF>(kc[j], q[t][j], acc);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &y = x[t][4 * sub + e];
                        if constexpr (!BF) y = __builtin_fmaf(par_offset<BF>(kp[e]), qsum[t][g], g ? y : 0.f);
                        y = __builtin_fmaf(par_step<BF>(kp[e]), acc[e], y);
                    }
                }
            }
        }
        if (masked) {
            asm volatile("");                    // (a branch, not sixteen selects in every tile)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (TREE) {
                    const uint32_t bits = tree_bits(t, tile);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[t][e] = bits >> (16 * (e >> 2) + (e & 3)) & 1 ? x[t][e] : -__builtin_inff();
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int slot = 32 * tile + 16 * (e >> 2) + 4 * b4 + (e & 3);
                    if (!((slot >= lo[t]) & (slot < hi[t]))) x[t][e] = -__builtin_inff();
                }
            }
        }
        float top[NT];
        bool move = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float m = fmaxf(x[t][0], x[t][1]);
#pragma unroll
            for (int e = 2; e < 8; ++e) m = fmaxf(m, x[t][e]);
            top[t] = BF ? m * c1 : __builtin_fmaf(m, c1, -lift[t]);
            move |= top[t] > ref[t] + kSlack;
        }
        const bool wide = !BF && __builtin_amdgcn_ballot_w64(steps > step_limit);
        const bool moves = __builtin_amdgcn_ballot_w64(move);
        if (moves || wide) {
            float by[NT] = {};                   // what each row's lift goes down by
            if (wide) {
                float met[NT];
                if (!masked) {                   // (neither infinities nor NaN)
                    const float all = lo_f32<BF>(max_lanes(steps < 0x7C00u ? steps : 0u));
#pragma unroll
                    for (int t = 0; t < NT; ++t) met[t] = all;
                } else {                         // each row looks at the slots that it sees
#pragma unroll
                    for (int t = 0; t < NT; ++t) met[t] = 0.f;
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float s = par_step<BF>(
                                lds_get<uint32_t>(params + 128 * (NG + g) + 64 * (e >> 2) + 4 * (e & 3)));
                            const int slot = 32 * tile + 16 * (e >> 2) + 4 * b4 + (e & 3);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                bool seen = (slot >= lo[t]) & (slot < hi[t]);
                                if constexpr (TREE) seen = tree_bits(t, tile) >> (16 * (e >> 2) + (e & 3)) & 1;
                                if (seen & (s < __builtin_inff())) met[t] = fmaxf(met[t], s);
                            }
                        }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        met[t] = fmaxf(met[t], __shfl_xor(met[t], 16));
                        met[t] = fmaxf(met[t], __shfl_xor(met[t], 32));
                    }
                }
                float highest = 0.f;
#pragma unroll
                for (int t = 0; t < NT; ++t) {   // a step in [2^(e - 1), 2^e): lift at most 14 - e, at least 0
                    const float to = fmaxf(fminf(lift[t], (float)(14 - __builtin_amdgcn_frexp_expf(met[t]))), 0.f);
                    by[t] = lift[t] - to;
                    lift[t] = to;
                    highest = fmaxf(highest, to);
                }
                step_limit = (29u - (uint32_t)__uint_as_float(max_lanes(__float_as_uint(highest)))) * 1024 - 1;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float m = fmaxf(top[t], __shfl_xor(top[t], 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                // (an infinite maximum stays out of the reference: its weight becomes infinite)
                m = fmaxf(ref[t], fminf(m, 3e38f));
                // (steps that a row does not see leave its last bits as they are)
                if (TREE && !moves) m = ref[t];
                if constexpr (!BF) m += by[t];
                const float f = __builtin_amdgcn_exp2f(ref[t] - m);
                ref[t] = m;
                sum[t] *= f;
                mids[t] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) psum[t][g] *= f;
#pragma unroll
                for (int o = 0; o < kOut; ++o) out[t][o] *= f;
            }
        }
        // weights, and their products with the values' steps as matrix operands
        u4 pr[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][e], c1, -ref[t]));
                sum[t] += x[t][e];
            }
            if constexpr (kMidRows)
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[t][e] = pack2<BF>(x[t][e], x[t][4 + e]);
        }
        if constexpr (kMidRows) {
            // sum_t p_t (m_t + 8 s_t) of all groups in two matrix products, row g of the first
            // operand holding group g: the rounded p_t with the middles in two parts
            const lds_u8 *mine = at + 2 * T::kCodes + 128 * (NG + (r < NG ? r : NG - 1)) + 16 * b4;
            const u4 p0 = lds_get<u4>(mine), p1 = lds_get<u4>(mine + 64);
            u4 high, low;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m0 = finite(__builtin_fmaf(8.0f, par_step<BF>(p0[e]), par_offset<BF>(p0[e])), kLargest<BF>);
                const float m1 = finite(__builtin_fmaf(8.0f, par_step<BF>(p1[e]), par_offset<BF>(p1[e])), kLargest<BF>);
                high[e] = pack2<BF>(m0, m1);
                low[e] = pack2<BF>(m0 - lo_f32<BF>(high[e]), m1 - hi_f32<BF>(high[e]));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mids[t] = mfma16x16x32_t<BF>(high, pr[t], mids[t]);
                mids[t] = mfma16x16x32_t<BF>(low, pr[t], mids[t]);
            }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const u4 p0 = lds_get<u4>(params + 128 * (NG + g)), p1 = lds_get<u4>(params + 128 * (NG + g) + 64);
            u4 pw[NT];
            float st[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) st[e] = par_step<BF>(e < 4 ? p0[e & 3] : p1[e & 3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float ps[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) ps[e] = mul_legacy(x[t][e], st[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) pw[t][e] = pack2<BF>(ps[e], ps[4 + e]);
                psum[t][g] = mfma16x16x32_t<BF>(ones, pw[t], psum[t][g]);
            }
            if constexpr (!kMidRows) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (of a seen slot's NaN, P_t is NaN)
                    const float mid = finite(
                        __builtin_fmaf(8.0f, st[e], par_offset<BF>(e < 4 ? p0[e & 3] : p1[e & 3])), kLargest<true>);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mids[t][0] = __builtin_fmaf(x[t][e], mid, mids[t][0]);
                }
            }
#pragma unroll
            for (int o = g * kBlocks; o < (g + 1) * kBlocks; ++o) {
                if constexpr (kBlocks >= 4) {
                    if (o % 4 == 0) {
                        const u4 words = lds_get<u4>(at + T::kCodes + 256 * o + 16 * lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const u4 vc = based_codes<BF>(words[i], cc);
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                out[t][o + i] = mfma16x16x32_t<BF>(vc, pw[t], out[t][o + i]);
                        }
                    }
                } else if (o % 2 == 0) {         // two words a group
                    const u2 words = lds_get<u2>(at + T::kCodes + 1024 * (o / 4) + 16 * lane + 4 * (o % 4));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const u4 vc = based_codes<BF>(words[i], cc);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            out[t][o + i] = mfma16x16x32_t<BF>(vc, pw[t], out[t][o + i]);
                    }
                }
            }
        }
    };

    int at_slot = 0;
    for (int tile = chunk0 + wave; tile < chunk1; tile += kWaves) {
        issue();
        wait_loads<(kRing - 1) * Copy::kLoads>();            // the oldest tile has landed
        __builtin_amdgcn_sched_barrier(0);
        if (there >> at_slot & 1) {
            const lds_u8 *at = lds + (wave * kRing + at_slot) * T::kBytes;
            step(tile, at);
        }
        at_slot = at_slot + 1 == kRing ? 0 : at_slot + 1;
        __builtin_amdgcn_sched_barrier(0);                   // its reads are done before a copy may overwrite it
    }
    wait_loads<0>();

    // join the waves: common reference, then the sums through LDS (which the tiles leave)
    lds_u8 *const refs = lds + Shape::kStats, *const sums = refs + 4 * kWaves * kRows;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sum[t] += __shfl_xor(sum[t], 16);
        sum[t] += __shfl_xor(sum[t], 32);
        if constexpr (!kMidRows) {
            mids[t][0] += __shfl_xor(mids[t][0], 16);
            mids[t][0] += __shfl_xor(mids[t][0], 32);
        }
        if (b4 == 0) {
            lds_put(refs + 4 * (wave * kRows + 16 * t + r), ref[t]);
            lds_put(sums + 4 * (wave * kRows + 16 * t + r), sum[t]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float m = lds_get<float>(refs + 4 * (16 * t + r));
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, lds_get<float>(refs + 4 * (i * kRows + 16 * t + r)));
        const float f = __builtin_amdgcn_exp2f(ref[t] - m);
        float mid[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g)         // row g of the product: register g % 4 of the lanes with b4 = g / 4
            mid[g] = kMidRows ? __shfl(mids[t][g % 4], 16 * (g / 4) + r) : mids[t][0];
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
            const int g = o / kBlocks;
            const f4 y = (out[t][o] - (kCodeBase<BF> + 8.0f) * psum[t][g] + mid[g]) * f;
            lds_put(lds + (wave * kRows + 16 * t + r) * Shape::kOutRow + 64 * o + 16 * b4, y);
        }
    }
    __syncthreads();
    const bool whole = w.t1 - w.t0 <= plan.chunk;       // this workgroup saw everything
    float *part = static_cast<float *>(a.workspace) +
                  (((int64_t)w.b * me.groups + me.group) * plan.chunks + me.chunk) * kRows * (D + 2);
    for (int idx = threadIdx.x; idx < kRows * (D / 4); idx += kThreads) {
        const int col = idx / (D / 4), d = 4 * (idx % (D / 4));
        const int row = w.row0 + col;
        if (row >= w.rows) break;
        float m = lds_get<float>(refs + 4 * col), total = 0.f;
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, lds_get<float>(refs + 4 * (i * kRows + col)));
        f4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            total += lds_get<float>(sums + 4 * (i * kRows + col)) *
                     __builtin_amdgcn_exp2f(lds_get<float>(refs + 4 * (i * kRows + col)) - m);
            y += lds_get<f4>(lds + (i * kRows + col) * Shape::kOutRow + 4 * d);
        }
        if (whole) {
            const int i = row / G;
            const int64_t at_q = w.first + i;
            const int head = w.h * G + row - i * G;
            const float inv = total == 0.f ? 0.f : 1.0f / total;
            *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at_q * a.out_stride + (int64_t)head * D + d) =
                pack4<BF>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            if (a.lse && d == 0)
                a.lse[at_q * a.q_heads + head] =
                    total == 0.f ? -__builtin_inff() : (m + __log2f(total)) * (1.0f / kLog2e);
        } else {
            *reinterpret_cast<f4 *>(part + col * D + d) = y;
            if (d == 0) {
                part[kRows * D + col] = m;
                part[kRows * D + kRows + col] = total;
            }
        }
    }
}

// Joins the chunks of one row: out = sum_c 2^(ref_c - ref) out_c / sum_c 2^(ref_c - ref) sum_c.
// D/4 lanes take four channels each; the other lanes of the workgroup take other chunks.
constexpr int kJoin = 256;
template <bool BF, int D>
__global__ void __launch_bounds__(kJoin) join_kernel(Kv4AttnArgs a, Plan plan) {
    constexpr int kLanes = D / 4, kSets = kJoin / kLanes;
    const int rows = plan.rows, kvh = a.c.kv_heads, G = a.q_heads / kvh;
    Work w;
    const int col = blockIdx.x;
    if (!work_of(a, blockIdx.z, blockIdx.y % kvh, (blockIdx.y / kvh) * rows, rows, &w)) return;
    const int row = w.row0 + col;
    if (row >= w.rows || w.t1 - w.t0 <= plan.chunk) return;
    const int chunks = (w.t1 - w.t0 + plan.chunk - 1) / plan.chunk;
    const int64_t step = (int64_t)rows * (D + 2);
    const float *part = static_cast<const float *>(a.workspace) +
                        ((int64_t)w.b * gridDim.y + blockIdx.y) * plan.chunks * step;
    const float *refs = part + rows * D + col, *sums = refs + rows;
    __shared__ float tops[kJoin / 64], totals[kSets];
    __shared__ f4 outs[kSets][kLanes];
    float m = kNone;
    for (int c = threadIdx.x; c < chunks; c += kJoin) m = fmaxf(m, refs[c * step]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoin / 64; ++i) m = fmaxf(m, tops[i]);
    const int set = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    float total = 0.f;
    f4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = set; c < chunks; c += kSets) {
        const float f = __builtin_amdgcn_exp2f(refs[c * step] - m);
        total += f * sums[c * step];
        y += f * *reinterpret_cast<const f4 *>(part + c * step + col * D + 4 * lane);
    }
    outs[set][lane] = y;
    if (lane == 0) totals[set] = total;
    __syncthreads();
    if (set > 0) return;
#pragma unroll
    for (int i = 1; i < kSets; ++i) {
        y += outs[i][lane];
        total += totals[i];
    }
    const int i = row / G, head = w.h * G + row - i * G;
    const int64_t at = w.first + i;
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at * a.out_stride + (int64_t)head * D + 4 * lane) =
        pack4<BF>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && lane == 0)
        a.lse[at * a.q_heads + head] = total == 0.f ? -__builtin_inff() : (m + __log2f(total)) * (1.0f / kLog2e);
}

// The same for trees, which have many rows: D/4 lanes take a whole row each, so that a workgroup joins
// 1024 / D of them (12 trees of 5 to 37 drafts over 900 to 12000 slots, four chunks: 21 us a row at a
// time, 6.5 here; 7 over 1000, six chunks: 4.3 and 6.1).
template <bool BF, int D>
__global__ void __launch_bounds__(kJoin) join_rows_kernel(Kv4AttnArgs a, Plan plan) {
    constexpr int kLanes = D / 4, kSets = kJoin / kLanes;
    const int rows = plan.rows, kvh = a.c.kv_heads, G = a.q_heads / kvh;
    Work w;
    const int col = blockIdx.x * kSets + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    if (!work_of(a, blockIdx.z, blockIdx.y % kvh, (blockIdx.y / kvh) * rows, rows, &w)) return;
    const int row = w.row0 + col;
    if (col >= rows || row >= w.rows || w.t1 - w.t0 <= plan.chunk) return;
    const int chunks = (w.t1 - w.t0 + plan.chunk - 1) / plan.chunk;
    const int64_t step = (int64_t)rows * (D + 2);
    const float *part = static_cast<const float *>(a.workspace) +
                        ((int64_t)w.b * gridDim.y + blockIdx.y) * plan.chunks * step;
    const float *refs = part + rows * D + col, *sums = refs + rows;
    float m = kNone, total = 0.f;
    f4 y = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < chunks; ++c) m = fmaxf(m, refs[c * step]);
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
        const float f = __builtin_amdgcn_exp2f(refs[c * step] - m);
        total += f * sums[c * step];
        y += f * *reinterpret_cast<const f4 *>(part + c * step + col * D + 4 * lane);
    }
    const int i = row / G, head = w.h * G + row - i * G;
    const int64_t at = w.first + i;
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at * a.out_stride + (int64_t)head * D + 4 * lane) =
        pack4<BF>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    if (a.lse && lane == 0)
        a.lse[at * a.q_heads + head] = total == 0.f ? -__builtin_inff() : (m + __log2f(total)) * (1.0f / kLog2e);
}

// Most chunks of a row that one set of lanes goes through, and the least workgroups of a row each from which it does.
constexpr int kJoinChunks = 16, kJoinMany = 4096;

template <typename F>
hipError_t by_shape(const Kv4Cache &c, F f) {
    auto typed = [&](auto d, auto ng) {
        return c.bf16 ? f(std::true_type{}, d, ng) : f(std::false_type{}, d, ng);
    };
    return kv4_dispatch(c.head_dim, c.groups, typed);
}

}  // namespace

int64_t kv4_attention_row_tiles(const Kv4AttnArgs &a) {
    return ((int64_t)rows_of(a) + tile_rows(a) - 1) / tile_rows(a);
}

int64_t kv4_tree_blocks(const Kv4AttnArgs &a) {
    const Plan p = plan_of(a);
    return (int64_t)a.c.kv_heads * p.row_tiles * p.chunks;
}

size_t kv4_attention_workspace_bytes(const Kv4AttnArgs &a) {
    const Plan p = plan_of(a);
    if (p.chunks <= 1) return 0;
    return (size_t)a.c.batch * a.c.kv_heads * p.row_tiles * p.chunks * p.rows * (a.c.head_dim + 2) * 4;
}

hipError_t launch_kv4_attention(const Kv4AttnArgs &a, hipStream_t stream) {
    const Plan p = plan_of(a);
    const dim3 grid((unsigned)p.chunks, (unsigned)(a.c.kv_heads * p.row_tiles), (unsigned)a.c.batch);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        if (rows_of(a) > kFewRows) {
            const hipError_t e = launch_kv4_prefill(a, p, stream);
            if (e != hipSuccess) return e;
        } else if (p.rows == 16) {
            if (a.tree)
                attend_kernel<bf(), d(), ng(), 1, true><<<tree_grid(a, p), kThreads, 0, stream>>>(a, p);
            else
                attend_kernel<bf(), d(), ng(), 1, false><<<grid, kThreads, 0, stream>>>(a, p);
        } else if constexpr (d() <= 128) {
            if (a.tree)
                attend_kernel<bf(), d(), ng(), 2, true><<<tree_grid(a, p), kThreads, 0, stream>>>(a, p);
            else
                attend_kernel<bf(), d(), ng(), 2, false><<<grid, kThreads, 0, stream>>>(a, p);
        }
        hipError_t e = hipGetLastError();
        const int64_t of_row = (int64_t)std::min(p.rows, rows_of(a)) * grid.y * grid.z;
        if (e == hipSuccess && p.chunks > 1 && a.tree && p.chunks <= kJoinChunks && of_row >= kJoinMany) {
            constexpr int kSets = 4 * kJoin / d();
            join_rows_kernel<bf(), d()>
                <<<dim3((std::min(p.rows, rows_of(a)) + kSets - 1) / kSets, grid.y, grid.z), kJoin, 0, stream>>>(a, p);
            e = hipGetLastError();
        } else if (e == hipSuccess && p.chunks > 1) {
            join_kernel<bf(), d()><<<dim3(std::min(p.rows, rows_of(a)), grid.y, grid.z), kJoin, 0, stream>>>(a, p);
            e = hipGetLastError();
        }
        return e;
    });
}

}  // namespace w4a16
