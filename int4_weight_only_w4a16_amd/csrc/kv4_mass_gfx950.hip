// The attention weight of every cached slot: for each key/value head
//   acc[t] += sum over the rows that see slot t of exp2(c1 q . k_t - lse log2(e)),
//   c1 = scale log2(e),
// rows being (new token, query head of the group) pairs.  Every slot has one
// owner, a lane group of one wave, and its rows come in one order, so the
// sums are the same bits each time.
//
// Few rows (a decode step): a wave walks over tiles with the rows' q in
// registers; keys are the exact operands B + c, steps and offsets act on the
// fp32 sums.  Reads the key half of the cache once, and is bound by that and
// by unpacking it.
//
// Many rows (a prompt): a wave keeps the keys of 32 slots in registers, as
// two 16-bit parts each (k = high + low to 2^-17 or better), and the rows
// pass by in LDS, 64 at a time, shared by the waves of up to eight such tiles.  Two products a
// channel block instead of one, but a weight then takes one fma, one
// exponential and one add.  Bound by the matrix cores.
//
// Measured: 8 sequences of 2000 to 16000 slots, one token, 40 heads on 8: 17 us (2.7 TB/s of the
// keys' half; the rest is the unpacking).  2048 tokens over 8191 slots, 32 heads on 8: 236 us, 490
// TFLOP/s of the formula's product and twice that with the low parts.

#include <algorithm>

#include "kv4_attn.hpp"

namespace w4a16 {
namespace {

// Sum over the 16 lanes of a row, in each of them.
__device__ __forceinline__ float sum16(float v) {
#define W4A16_ROR(N) \
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + N, 0xF, 0xF, true))
    W4A16_ROR(8);
    W4A16_ROR(4);
    W4A16_ROR(2);
    W4A16_ROR(1);
#undef W4A16_ROR
    return v;
}

// The key half of a tile, copied to LDS without passing through registers.
template <int D, int NG>
struct KeyCopy {
    using T = Tile<D, NG>;
    static constexpr int kParams = NG <= 2 ? 256 : 128 * NG;         // (256 bytes an instruction)
    static constexpr int kBytes = T::kCodes + kParams;
    static constexpr int kLoads = D / 64 + kParams / 256;
    static __device__ __forceinline__ void issue(const uint8_t *tile, uint32_t bytes, lds_u8 *to, int lane) {
        const auto rsrc = make_rsrc(tile, bytes);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + 1024 * j), 16, 16 * lane, 1024 * j, 0, 0);
#pragma unroll
        for (int j = 0; j < kParams / 256; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + T::kCodes + 256 * j), 4, 4 * lane,
                                                     2 * T::kCodes + 256 * j, 0, 0);
    }
};

template <bool BF, int D, int NG, int NT>
__global__ void __launch_bounds__(kThreads) few_rows_kernel(Kv4AttnArgs a, int chunk) {
    using T = Tile<D, NG>;
    using Copy = KeyCopy<D, NG>;
    constexpr int kSteps = D / 32, kPer = kSteps / NG, kRing = 3;
    __shared__ __align__(16) uint8_t lds_raw[kWaves * kRing * Copy::kBytes];
    lds_u8 *const lds = (lds_u8 *)lds_raw;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, b4 = lane >> 4;
    const int tpp = a.c.tiles_per_page, kvh = a.c.kv_heads, G = a.q_heads / kvh;
    auto load_ids = [&](int tile) {
        const int at = tile / tpp + lane;
        return at < a.c.table_stride ? a.c.table[(int64_t)blockIdx.z * a.c.table_stride + at] : -1;
    };
    int ids = load_ids((int)blockIdx.x * chunk);
    Work w;
    if (!work_of(a, blockIdx.z, blockIdx.y, 0, 16 * NT, &w)) return;
    const int chunk0 = w.t0 + (int)blockIdx.x * chunk, chunk1 = min(chunk0 + chunk, w.t1);
    if (chunk0 >= w.t1) return;
    const int page0 = chunk0 / tpp;
    if (w.t0 > 0) ids = load_ids(chunk0);
    int next = chunk0 + wave, page = 0, in = chunk0 - page0 * tpp + wave, slot_next = 0;
    uint32_t there = 0;
    auto issue = [&]() {
        while (in >= tpp) {
            in -= tpp;
            ++page;
        }
        const int id = next < chunk1 ? __builtin_amdgcn_readlane(ids, page) : -1;
        const bool ok = (unsigned)id < (unsigned)a.c.num_pages;
        const uint8_t *p = a.c.pages + (((int64_t)(ok ? id : 0) * kvh + w.h) * tpp + in) * T::kBytes;
        Copy::issue(p, ok ? T::kBytes : 0, lds + (wave * kRing + slot_next) * Copy::kBytes, lane);
        there = (there & ~(1u << slot_next)) | ((ok ? 1u : 0u) << slot_next);
        slot_next = slot_next + 1 == kRing ? 0 : slot_next + 1;
        next += kWaves;
        in += kWaves;
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue();

    u4 q[NT][kSteps];
    float qsum[NT][NG], shift[NT];
    f4 init[NT][NG];
    int lo[NT], hi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = 16 * t + r;
        const bool in_seq = row < w.rows;
        const int i = in_seq ? row / G : 0, head = w.h * G + (in_seq ? row - i * G : 0);
        const int64_t token = w.first + i;
        const float lse = a.lse[token * a.q_heads + head];
        // (a row that saw nothing adds nothing)
        const bool seen = in_seq && lse != -__builtin_inff();
        lo[t] = seen ? row_lo(i, w.start, a.window) : 0;
        hi[t] = seen ? row_hi(i, w.start, w.len, a.causal) : 0;
        shift[t] = -lse * kLog2e;
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + token * a.q_stride + (int64_t)head * D + 8 * b4;
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
    }
    const float c1 = a.scale * kLog2e;
    const CodeConsts cc = code_consts<BF>();
    float *const acc = a.acc + ((int64_t)w.b * kvh + w.h) * a.acc_stride;

    int at_slot = 0;
    for (int tile = chunk0 + wave; tile < chunk1; tile += kWaves) {
        // lane r < 8 of block b4 adds to slot 16 (r / 4) + 4 b4 + r % 4
        const int mine = 32 * tile + 16 * (r >> 2) + 4 * b4 + (r & 3);
        const bool writes = r < 8 && mine < w.len;
        float before = 0.f;
        if (writes) before = acc[mine];
        issue();
        wait_loads<(kRing - 1) * Copy::kLoads>();
        __builtin_amdgcn_sched_barrier(0);
        if (there >> at_slot & 1) {
            const lds_u8 *at = lds + (wave * kRing + at_slot) * Copy::kBytes;
            const lds_u8 *params = at + T::kCodes + 16 * b4;
            float mass[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
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
                u4 kp[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) kp[g] = lds_get<u4>(params + 128 * g + 64 * sub);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        f4 s = init[t][g];
#pragma unroll
                        for (int j = g * kPer; j < (g + 1) * kPer; ++j) s = mfma16x16x32_t<BF>(kc[j], q[t][j], s);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = __builtin_fmaf(par_step<BF>(kp[g][e]), s[e],
                                                  __builtin_fmaf(par_offset<BF>(kp[g][e]), qsum[t][g], x[e]));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int slot = 32 * tile + 16 * sub + 4 * b4 + e;
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c1, shift[t]));
                        mass[4 * sub + e] += (slot >= lo[t]) & (slot < hi[t]) ? p : 0.f;
                    }
                }
            }
            float add = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float total = sum16(mass[e]);
                add = r == e ? total : add;
            }
            if (writes) acc[mine] = before + add;
        }
        at_slot = at_slot + 1 == kRing ? 0 : at_slot + 1;
        __builtin_amdgcn_sched_barrier(0);                   // its reads are done before a copy may overwrite it
    }
    wait_loads<0>();
}

// ---- many rows ----

// How many waves share a tile of slots: with two, each takes the other 32 rows of a stage, so that
// the waves on a SIMD cover each other's exponentials and products (256 channels: the keys'
// registers allow one).
constexpr int kStageRows = 64;
template <int D>
constexpr int kSplit = D <= 128 ? 2 : 1;
template <int D, int TILES>
constexpr int kManyThreads = 64 * TILES * kSplit<D>;

// TILES: tiles of slots of a workgroup.
template <bool BF, int D, int NG, int TILES>
__global__ void __launch_bounds__((kManyThreads<D, TILES>)) many_rows_kernel(Kv4AttnArgs a) {
    using T = Tile<D, NG>;
    constexpr int kManyTiles = TILES, kManySlots = 32 * TILES;
    constexpr int kManyWaves = kManyThreads<D, TILES> / 64;
    constexpr int kDeep = D / 16;                                // 16-channel products
    constexpr int kStageBytes = kStageRows * D * 2, kRing = 3;
    constexpr int kCopies = kStageBytes / 1024 < kManyWaves ? 1 : kStageBytes / 1024 / kManyWaves;   // KiB that a wave copies
    constexpr int kHandover = kSplit<D> > 1 ? 4096 * kManyTiles : 0;
    __shared__ __align__(16) uint8_t lds_raw[kRing * kStageBytes > kHandover ? kRing * kStageBytes : kHandover];
    lds_u8 *const lds = (lds_u8 *)lds_raw;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int kvh = a.c.kv_heads, G = a.q_heads / kvh;
    Work w;
    if (!work_of(a, blockIdx.z, blockIdx.y, 0, 0x3fffffff, &w)) return;
    const int tile0 = w.t0 + (int)blockIdx.x * kManyTiles, tile = tile0 + wave % kManyTiles;
    if (tile0 >= w.t1) return;
    const uint8_t *const p =
        tile < w.t1 ? tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, w.b, w.h, tile) : nullptr;

    // the rows that see any of the workgroup's slots, in stages of kStageRows from a multiple of it
    const int i0 = a.causal ? max(0, 32 * tile0 - w.start) : 0;
    const int64_t last_slot = 32 * (int64_t)tile0 + kManySlots - 1;
    const int i1 = a.window > 0 ? (int)min((int64_t)w.n, last_slot + a.window - w.start) : w.n;
    const int row_begin = i0 * G / kStageRows * kStageRows;
    const int row_end = min((int64_t)i1 * G, (int64_t)w.rows);
    if (row_begin >= row_end) return;

    // Where a row's q and lse lie, for one row a lane that advances by a stage at a time: no
    // division in the loop.  A row past the last stands for the last.
    const int step_token = kStageRows / G, step_head = kStageRows % G;
    const uint16_t *const q0 = static_cast<const uint16_t *>(a.q) + (int64_t)w.first * a.q_stride + (int64_t)w.h * G * D;
    const float *const lse0 = a.lse + (int64_t)w.first * a.q_heads + w.h * G;
    struct Row {
        int row, token, head;
    };
    auto row_at = [&](int row) { return Row{row, row / G, row % G}; };
    auto advance = [&](Row &x) {
        x.row += kStageRows;
        x.token += step_token;
        x.head += step_head;
        if (x.head >= G) {
            x.head -= G;
            ++x.token;
        }
    };
    const int last_token = w.n - 1, last_head = G - 1;
    auto q_of = [&](const Row &x) {
        const bool in = x.row < w.rows;
        return q0 + (int64_t)(in ? x.token : last_token) * a.q_stride + (in ? x.head : last_head) * D;
    };
    auto lse_of = [&](const Row &x) {
        const bool in = x.row < w.rows;
        return lse0[(int64_t)(in ? x.token : last_token) * a.q_heads + (in ? x.head : last_head)];
    };

    // a stage: 16-channel blocks of 32 rows, a KiB each, as matrix operands.  Copy i of this wave
    // is block u % kDeep of the 32 rows u / kDeep, u = wave + waves * i.
    Row copy_row[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
        copy_row[i] = row_at(row_begin + 32 * ((wave + kManyWaves * i) % (kStageBytes / 1024) / kDeep) + col);
    auto copy = [&](int slot) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int unit = (wave + kManyWaves * i) % (kStageBytes / 1024), j = unit % kDeep;
            const uint16_t *src = q_of(copy_row[i]) + 16 * j + 8 * half;
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<const __attribute__((address_space(1))) void *>(reinterpret_cast<uintptr_t>(src)),
                (lds_void *)(lds + slot * kStageBytes + 1024 * unit), 16, 0, 0);
            advance(copy_row[i]);
        }
    };
    int slot_next = 0;
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
        copy(slot_next);
        slot_next = slot_next + 1 == kRing ? 0 : slot_next + 1;
    }

    // this wave's 32 keys in two parts: row `col` of the operands, channels 16 j + 8 half + 0..7
    u4 high[kDeep], low[kDeep];
    {
        uint32_t words[kDeep] = {}, pars[NG] = {};
        if (p) {
#pragma unroll
            for (int j = 0; j < kDeep; ++j) words[j] = reinterpret_cast<const uint32_t *>(p)[key_word<D>(col, 2 * j + half)];
#pragma unroll
            for (int g = 0; g < NG; ++g) pars[g] = reinterpret_cast<const uint32_t *>(p + 2 * T::kCodes)[32 * g + col];
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const float st = par_step<BF>(pars[16 * j / T::kGroup]), off = par_offset<BF>(pars[16 * j / T::kGroup]);
            uint32_t even = words[j] & 0x0F0F0F0Fu, odd = (words[j] >> 4) & 0x0F0F0F0Fu;
            asm("" : "+v"(even), "+v"(odd));
#pragma unroll
            for (int e = 0; e < 4; ++e) {        // channels 2 e and 2 e + 1: nibbles e and e + 4
                const uint32_t src = e & 1 ? odd : even;
                const float k0 = fminf(__builtin_fmaf(st, ubyte_f32(src, e >> 1), off), kLargest<BF>);
                const float k1 = fminf(__builtin_fmaf(st, ubyte_f32(src, 2 + (e >> 1)), off), kLargest<BF>);
                high[j][e] = pack2<BF>(k0, k1);
                low[j][e] = pack2<BF>(k0 - lo_f32<BF>(high[j][e]), k1 - hi_f32<BF>(high[j][e]));
            }
        }
    }

    const float c1 = a.scale * kLog2e;
    const f16v zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    f16v mass = zero;
    // lse of this lane's columns, loaded a stage ahead
    constexpr int kLse = 2 / kSplit<D>;
    float lse[kLse], lse_next[kLse];
    Row lse_row[kLse];
#pragma unroll
    for (int step = 0; step < kLse; ++step)
        lse_row[step] = row_at(row_begin + 32 * (kSplit<D> > 1 ? wave / kManyTiles : step) + col);
    auto load_lse = [&]() {
#pragma unroll
        for (int step = 0; step < kLse; ++step) {
            lse_next[step] = lse_of(lse_row[step]);
            advance(lse_row[step]);
        }
    };
    load_lse();
    // rows that see the whole tile: [all0, all1)
    const int64_t first_all = a.causal ? max(0, 32 * tile + 31 - w.start) : 0;
    const int64_t last_all = a.window > 0 ? min((int64_t)w.n, (int64_t)32 * tile + a.window - w.start) : w.n;
    const bool any_all = 32 * tile + 32 <= w.len;
    const int all0 = any_all ? (int)min(first_all * G, (int64_t)w.rows) : w.rows;
    const int all1 = any_all ? (int)max(last_all * G, (int64_t)0) : 0;
    int at_slot = 0;
    for (int row0 = row_begin; row0 < row_end; row0 += kStageRows) {
#pragma unroll
        for (int step = 0; step < kLse; ++step) lse[step] = lse_next[step];
        load_lse();
        copy(slot_next);
        slot_next = slot_next + 1 == kRing ? 0 : slot_next + 1;
        wait_loads<(kRing - 1) * kCopies + kLse>();              // this wave's share of the oldest stage is there
        lds_barrier();                                           // ... and the others'
        const lds_u8 *const at = lds + at_slot * kStageBytes + 16 * lane;
#pragma unroll
        for (int step = 0; step < 2 / kSplit<D>; ++step) {
            const int s = kSplit<D> > 1 ? wave / kManyTiles : step;
            const int ra = row0 + 32 * s, rb = ra + 31;          // the rows of this product
            f16v x = zero;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                const u4 q = lds_get<u4>(at + 1024 * (kDeep * s + j));
                x = mfma32x32x16_t<BF>(high[j], q, x);
                x = mfma32x32x16_t<BF>(low[j], q, x);
            }
            const float shift = lse[step] == -__builtin_inff() ? lse[step] : -lse[step] * kLog2e;
            const bool all = ra >= all0 && rb < all1;
            if (all) {
#pragma unroll
                for (int i = 0; i < 16; ++i) mass[i] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], c1, shift));
            } else {
                const int row = ra + col, i = min(row, w.rows - 1) / G;
                const bool in_seq = row < w.rows;
                int lo = (in_seq ? row_lo(i, w.start, a.window) : 0) - 32 * tile - 4 * half;
                int hi = (in_seq ? row_hi(i, w.start, w.len, a.causal) : 0) - 32 * tile - 4 * half;
                if (!in_seq) hi = lo;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int slot = 8 * (e >> 2) + (e & 3);
                    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c1, shift));
                    mass[e] += (slot >= lo) & (slot < hi) ? y : 0.f;
                }
            }
        }
        at_slot = at_slot + 1 == kRing ? 0 : at_slot + 1;
        lds_barrier();                                           // the stage may be overwritten
    }
    wait_loads<0>();
    // the tile's other wave hands its sums over in LDS, which the stages leave
    if constexpr (kSplit<D> > 1) {
        lds_barrier();
        lds_u8 *const mine = lds + (wave % kManyTiles) * 4096 + 16 * lane;
        if (wave >= kManyTiles)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lds_put(mine + 1024 * i, f4{mass[4 * i], mass[4 * i + 1], mass[4 * i + 2], mass[4 * i + 3]});
        lds_barrier();
        if (wave >= kManyTiles) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f4 v = lds_get<f4>(mine + 1024 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) mass[4 * i + e] += v[e];
        }
    }
    if (!p) return;
    // register e: slot 8 (e / 4) + 4 half + e % 4, summed over the 32 columns
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float v = sum16(mass[e]);
        v += __shfl_xor(v, 16);
        const int slot = 32 * tile + 8 * (e >> 2) + 4 * half + (e & 3);
        if (col == e && slot < w.len) {
            float *to = a.acc + ((int64_t)w.b * kvh + w.h) * a.acc_stride + slot;
            *to += v;
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

hipError_t launch_kv4_mass(const Kv4AttnArgs &a, hipStream_t stream) {
    const int rows = a.q_heads / a.c.kv_heads * a.max_q;
    int tiles = (a.max_kv + 31) / 32;
    if (a.window > 0) tiles = std::min<int64_t>(tiles, ((int64_t)a.window + a.max_q) / 32 + 2);
    const unsigned heads = (unsigned)a.c.kv_heads, batch = (unsigned)a.c.batch;
    // up to 64 rows fit the registers of the kernel for few (32 sequences of 4000 slots, 8 heads: 64
    // rows 57 us there and 174 here, of one sequence of 16000 slots 12 and 24)
    if (rows > 64) {
        // Eight tiles share a stage of rows, or fewer where half of the 256 CUs would be without
        // work (1600 rows, 8 heads of 128 channels, us with 8, 4 and 2: 8000 slots 55, 66 and 86;
        // 4000 slots 55, 38 and 39; 2000 slots 52, 35 and 31.  256 channels, 2000 slots: 83, 65, 78)
        auto go = [&](auto n) {
            const dim3 grid((unsigned)((tiles + n() - 1) / n()), heads, batch);
            return by_shape(a.c, [&](auto bf, auto d, auto ng) {
                many_rows_kernel<bf(), d(), ng(), n()><<<grid, kManyThreads<d(), n()>, 0, stream>>>(a);
                return hipGetLastError();
            });
        };
        const int64_t all = (int64_t)tiles * heads * batch;
        return all > 8 * 128                              ? go(std::integral_constant<int, 8>{})
               : all > 4 * 128 || a.c.head_dim > 128 ? go(std::integral_constant<int, 4>{})
                                                          : go(std::integral_constant<int, 2>{});
    }
    // chunks as the attention's, within the page ids that a wave holds (8 sequences of 2000 to
    // 16000 slots: 24.5 us with 512 workgroups, 18.3 with 1536, 22 with 2048)
    const int64_t want = std::max<int64_t>(1, (batch <= 4 ? 768 : 1536) / ((int64_t)heads * batch));
    const int chunk = chunk_of(a.c, tiles, want);
    const dim3 grid((unsigned)((tiles + chunk - 1) / chunk), heads, batch);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        if (rows <= 16)
            few_rows_kernel<bf(), d(), ng(), 1><<<grid, kThreads, 0, stream>>>(a, chunk);
        else if (rows <= 32)
            few_rows_kernel<bf(), d(), ng(), 2><<<grid, kThreads, 0, stream>>>(a, chunk);
        else
            few_rows_kernel<bf(), d(), ng(), 4><<<grid, kThreads, 0, stream>>>(a, chunk);
        return hipGetLastError();
    });
}

}  // namespace w4a16
