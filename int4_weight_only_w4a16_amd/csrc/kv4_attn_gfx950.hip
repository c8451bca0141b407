// Softmax attention over the 4-bit key/value cache.
//
// Rows are (new token, query head of the group) pairs; for row q and slot t
//   x_t = q . k_t,  k_t = m + s c per group of channels
//       = sum_g s_g (q_g . (16 + c_g)) + (m_g - 16 s_g) sum(q_g)
//   p_t = exp2(scale log2(e) x_t - ref),  out = sum_t p_t v_t / sum_t p_t,
//   sum_t p_t v_t = sum_t P_t (16 + c_t) - 24 sum_t P_t + sum_t p_t (m_t + 8 s_t),
//   P_t = p_t s_t rounded to the activation type.
// The codes go into the matrix instructions as the exact 16-bit numbers
// 16 + c; steps and offsets act on the fp32 sums.  The sum of the P_t comes
// from one more matrix product with ones, of the same rounded P_t, so that
// the 24 comes off exactly and only P_t (c_t - 8) feels their rounding.
// ref is a running reference per row, moved only when a tile's maximum
// passes it by more than kSlack: p_t stays below 2^kSlack, and P_t below
// 2^kSlack * (2 * 65504 / 15), which fp16 holds.

#include <algorithm>

#include "kv4_device.hpp"

namespace w4a16 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kSlack = 2.0f;
constexpr float kNone = -3e38f;        // reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;

// What a workgroup works on: a tile of rows of one head of one sequence, and
// a range of its slots.
struct Work {
    int b, h, len, n, first;      // sequence, head, slots, new tokens, row of q of the first new token
    int row0, rows;               // first row of the tile; rows of the sequence
    int t0, t1;                   // tiles of slots that any row of the tile sees
};

__device__ __forceinline__ bool work_of(const Kv4AttnArgs &a, int b, int h, int row0, int rows_per, Work *w) {
    const int64_t first = a.cu[b];
    const int64_t n64 = min((int64_t)a.cu[b + 1], a.T) - first;
    if (first < 0 || n64 <= 0) return false;
    w->b = b;
    w->h = h;
    w->first = (int)first;
    w->n = (int)min(n64, (int64_t)a.max_q);
    const int64_t cap = (int64_t)a.c.table_stride * a.c.tiles_per_page * 32;
    w->len = (int)min((int64_t)min(max(a.kv_len[b], 0), a.max_kv), cap);
    const int G = a.q_heads / a.c.kv_heads;
    w->row0 = row0;
    w->rows = w->n * G;
    if (row0 >= w->rows) return false;
    const int last = min(row0 + rows_per, w->rows) - 1;
    const int lo = row_lo(row0 / G, w->n, w->len, a.window);
    const int hi = row_hi(last / G, w->n, w->len, a.causal);
    w->t0 = lo >> 5;
    w->t1 = hi > lo ? (hi + 31) >> 5 : w->t0;
    return true;
}

// Rows per tile of rows: 16 NT.  Partial results of one (sequence, head, tile
// of rows, chunk): 16 NT x (D sums, reference, sum of p).
struct Plan {
    int nt, row_tiles, chunk, chunks;      // chunk: tiles of slots a workgroup takes
};

constexpr int kPlanSlots = 256 * 3;      // workgroups the chip holds at a time

Plan plan_of(const Kv4AttnArgs &a) {
    Plan p;
    const int rows = a.q_heads / a.c.kv_heads * a.max_q;
    p.nt = rows > 16 && a.c.head_dim <= 128 ? 2 : 1;      // (256 channels: two would not fit the registers)
    p.row_tiles = (rows + 16 * p.nt - 1) / (16 * p.nt);
    int tiles = (a.max_kv + 31) / 32;
    if (a.window > 0) tiles = std::min(tiles, (a.window + a.max_q) / 32 + 2);
    const int64_t groups = (int64_t)a.c.batch * a.c.kv_heads * p.row_tiles;
    const int64_t want = std::max<int64_t>(1, kPlanSlots / groups);
    p.chunk = (int)std::max<int64_t>(kWaves, (tiles + want - 1) / want);
    p.chunk = (p.chunk + kWaves - 1) / kWaves * kWaves;
    p.chunks = std::max(1, (tiles + p.chunk - 1) / p.chunk);
    return p;
}

template <int D, int NG>
struct Stage {
    u4 k[D / 64], v[D / 64];
    uint32_t par[NG];
    bool there;
};

template <bool BF, int D, int NG, int NT>
__global__ void __launch_bounds__(kThreads) attend_kernel(Kv4AttnArgs a, Plan plan) {
    using T = Tile<D, NG>;
    constexpr int kSteps = D / 32;            // 32-channel products of a slot
    constexpr int kPer = kSteps / NG;         // of them per group
    constexpr int kRows = 16 * NT;
    constexpr int kOut = D / 16;              // 16-channel blocks of the output
    constexpr int kBlocks = kOut / NG;        // of them per group
    struct Shared {
        __align__(16) uint32_t par[kWaves][64 * NG];
        float ref[kWaves][kRows], sum[kWaves][kRows];
        float out[kWaves][kRows][D + 4];
    };
    __shared__ Shared sh;

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, b4 = lane >> 4;
    Work w;
    const int kvh = a.c.kv_heads;
    if (!work_of(a, blockIdx.z, blockIdx.y % kvh, (blockIdx.y / kvh) * kRows, kRows, &w)) return;
    const int chunk0 = w.t0 + (int)blockIdx.x * plan.chunk;
    const int chunk1 = min(chunk0 + plan.chunk, w.t1);
    if (blockIdx.x > 0 && chunk0 >= w.t1) return;
    const int G = a.q_heads / kvh;

    // this lane's columns: NT rows of q, their channels as matrix operands, and what they see
    u4 q[NT][kSteps];
    f4 init[NT][NG];
    float qsum[NT][NG];
    int lo[NT], hi[NT];
    int all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = w.row0 + 16 * t + r;
        const bool there = row < w.rows;
        const int i = there ? row / G : 0;
        lo[t] = there ? row_lo(i, w.n, w.len, a.window) : 0;
        hi[t] = there ? row_hi(i, w.n, w.len, a.causal) : 0;
        if (there) {
            all_lo = max(all_lo, lo[t]);
            all_hi = min(all_hi, hi[t]);
        }
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + (int64_t)(w.first + i) * a.q_stride +
                              (int64_t)(w.h * G + (there ? row - i * G : 0)) * D + 8 * b4;
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
            const float z = -16.0f * qsum[t][g];
            init[t][g] = f4{z, z, z, z};
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
    float ref[NT], sum[NT], corr[NT][NG];
    f4 out[NT][kOut], psum[NT][NG];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        ref[t] = kNone;
        sum[t] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            corr[t][g] = 0.f;
            psum[t][g] = f4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int o = 0; o < kOut; ++o) out[t][o] = f4{0.f, 0.f, 0.f, 0.f};
    }

    auto load = [&](int tile, Stage<D, NG> &s) {
        s.there = false;
        if (tile >= chunk1) return;
        const uint8_t *p = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, w.b, w.h, tile);
        if (!p) return;
        s.there = true;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            s.k[j] = *reinterpret_cast<const u4 *>(p + 1024 * j + 16 * lane);
            s.v[j] = *reinterpret_cast<const u4 *>(p + T::kCodes + 1024 * j + 16 * lane);
        }
        const uint32_t *par = reinterpret_cast<const uint32_t *>(p + 2 * T::kCodes);
#pragma unroll
        for (int j = 0; j < NG; ++j) s.par[j] = par[64 * j + lane];
    };

    auto step = [&](int tile, const Stage<D, NG> &s) {
        // parameters: one load of the tile's words, then broadcasts out of LDS (a wave's own
        // area; its LDS operations are in order)
#pragma unroll
        for (int j = 0; j < NG; ++j) sh.par[wave][64 * j + lane] = s.par[j];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const u4 *par = reinterpret_cast<const u4 *>(sh.par[wave]);
        float x[NT][8];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            u4 kc[kSteps];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const int word = sub * kSteps + j;
                kc[j] = codes16<BF>(s.k[word >> 2][word & 3], cc);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const u4 kp = par[8 * g + 4 * sub + b4];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f4 acc = init[t][g];
#pragma unroll
                    for (int j = g * kPer; j < (g + 1) * kPer; ++j) acc = mfma16x16x32_t<BF>(kc[j], q[t][j], acc);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float m = par_offset<BF>(kp[e]), st = par_step<BF>(kp[e]);
                        float &y = x[t][4 * sub + e];
                        y = g == 0 ? m * qsum[t][0] : __builtin_fmaf(m, qsum[t][g], y);
                        y = __builtin_fmaf(st, acc[e], y);
                    }
                }
            }
        }
        const int base = 32 * tile;
        const bool masked = base < all_lo || base + 32 > all_hi;      // the same in every lane
        uint32_t see[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            see[t] = 0xFFu;
            if (masked) {
                see[t] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int slot = base + 16 * (e >> 2) + 4 * b4 + (e & 3);
                    const bool ok = slot >= lo[t] && slot < hi[t];
                    see[t] |= (ok ? 1u : 0u) << e;
                    if (!ok) x[t][e] = -__builtin_inff();
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
            top[t] = m * c1;
            move |= top[t] > ref[t] + kSlack;
        }
        if (__builtin_amdgcn_ballot_w64(move)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float m = fmaxf(top[t], __shfl_xor(top[t], 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                // (an infinite maximum stays out of the reference: its weight becomes infinite)
                m = fmaxf(ref[t], fminf(m, 3e38f));
                const float f = __builtin_amdgcn_exp2f(ref[t] - m);
                ref[t] = m;
                sum[t] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    corr[t][g] *= f;
                    psum[t][g] *= f;
                }
#pragma unroll
                for (int o = 0; o < kOut; ++o) out[t][o] *= f;
            }
        }
        // weights, and their products with the values' steps as matrix operands
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][e], c1, -ref[t]));
                sum[t] += x[t][e];
            }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const u4 p0 = par[8 * NG + 8 * g + b4], p1 = par[8 * NG + 8 * g + 4 + b4];
            float st[8], mid[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t p = e < 4 ? p0[e & 3] : p1[e & 3];
                st[e] = par_step<BF>(p);
                mid[e] = __builtin_fmaf(8.0f, st[e], par_offset<BF>(p));
            }
            u4 pw[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float ps[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float m = mid[e];
                    ps[e] = x[t][e] * st[e];
                    if (masked && !(see[t] >> e & 1)) ps[e] = m = 0.f;     // unseen: whatever is stored there
                    corr[t][g] = __builtin_fmaf(x[t][e], m, corr[t][g]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) pw[t][e] = pack2<BF>(ps[e], ps[4 + e]);
                psum[t][g] = mfma16x16x32_t<BF>(ones, pw[t], psum[t][g]);
            }
#pragma unroll
            for (int o = g * kBlocks; o < (g + 1) * kBlocks; ++o) {
                const u4 vc = codes16<BF>(s.v[o >> 2][o & 3], cc);
#pragma unroll
                for (int t = 0; t < NT; ++t) out[t][o] = mfma16x16x32_t<BF>(vc, pw[t], out[t][o]);
            }
        }
    };

    Stage<D, NG> s0, s1;
    int tile = chunk0 + wave;
    load(tile, s0);
    while (tile < chunk1) {
        load(tile + kWaves, s1);
        if (s0.there) step(tile, s0);
        tile += kWaves;
        if (tile >= chunk1) break;
        load(tile + kWaves, s0);
        if (s1.there) step(tile, s1);
        tile += kWaves;
    }

    // join the waves: common reference, then the sums through LDS
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sum[t] += __shfl_xor(sum[t], 16);
        sum[t] += __shfl_xor(sum[t], 32);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            corr[t][g] += __shfl_xor(corr[t][g], 16);
            corr[t][g] += __shfl_xor(corr[t][g], 32);
        }
        if (b4 == 0) {
            sh.ref[wave][16 * t + r] = ref[t];
            sh.sum[wave][16 * t + r] = sum[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float m = sh.ref[0][16 * t + r];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, sh.ref[i][16 * t + r]);
        const float f = __builtin_amdgcn_exp2f(ref[t] - m);
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
            const int g = o / kBlocks;
            const f4 y = (out[t][o] - 24.0f * psum[t][g] + corr[t][g]) * f;
            *reinterpret_cast<f4 *>(&sh.out[wave][16 * t + r][16 * o + 4 * b4]) = y;
        }
    }
    __syncthreads();
    const bool whole = w.t1 - w.t0 <= plan.chunk;       // this workgroup saw everything
    float *part = static_cast<float *>(a.workspace) +
                  (((int64_t)w.b * gridDim.y + blockIdx.y) * plan.chunks + blockIdx.x) * kRows * (D + 2);
    for (int at = threadIdx.x; at < kRows * (D / 4); at += kThreads) {
        const int col = at / (D / 4), d = 4 * (at % (D / 4));
        const int row = w.row0 + col;
        if (row >= w.rows) break;
        float m = sh.ref[0][col], total = 0.f;
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, sh.ref[i][col]);
        f4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            total += sh.sum[i][col] * __builtin_amdgcn_exp2f(sh.ref[i][col] - m);
            y += *reinterpret_cast<const f4 *>(&sh.out[i][col][d]);
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
template <bool BF, int D>
__global__ void __launch_bounds__(D) join_kernel(Kv4AttnArgs a, Plan plan) {
    const int kRows = 16 * plan.nt, kvh = a.c.kv_heads, G = a.q_heads / kvh;
    Work w;
    const int col = blockIdx.x;
    if (!work_of(a, blockIdx.z, blockIdx.y % kvh, (blockIdx.y / kvh) * kRows, kRows, &w)) return;
    const int row = w.row0 + col;
    if (row >= w.rows || w.t1 - w.t0 <= plan.chunk) return;
    const int chunks = (w.t1 - w.t0 + plan.chunk - 1) / plan.chunk;
    const float *part = static_cast<const float *>(a.workspace) +
                        ((int64_t)w.b * gridDim.y + blockIdx.y) * plan.chunks * kRows * (D + 2);
    const int64_t step = (int64_t)kRows * (D + 2);
    float m = kNone;
    for (int c = 0; c < chunks; ++c) m = fmaxf(m, part[c * step + kRows * D + col]);
    float total = 0.f, y = 0.f;
    for (int c = 0; c < chunks; ++c) {
        const float f = __builtin_amdgcn_exp2f(part[c * step + kRows * D + col] - m);
        total += f * part[c * step + kRows * D + kRows + col];
        y += f * part[c * step + col * D + threadIdx.x];
    }
    const int i = row / G, head = w.h * G + row - i * G;
    const int64_t at = w.first + i;
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    static_cast<uint16_t *>(a.out)[at * a.out_stride + (int64_t)head * D + threadIdx.x] =
        (uint16_t)pack2<BF>(y * inv, 0.f);
    if (a.lse && threadIdx.x == 0)
        a.lse[at * a.q_heads + head] = total == 0.f ? -__builtin_inff() : (m + __log2f(total)) * (1.0f / kLog2e);
}

// acc[b, h, t] += sum over the rows of head h of exp(scale q . k_t - lse): a
// wave owns a tile of slots, so every sum has one owner and one order.
template <bool BF, int D, int NG>
__global__ void __launch_bounds__(kThreads) mass_kernel(Kv4AttnArgs a) {
    using T = Tile<D, NG>;
    constexpr int kSteps = D / 32, kPer = kSteps / NG;
    __shared__ __align__(16) uint32_t shared[kWaves][32 * NG];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, b4 = lane >> 4;
    Work w;
    if (!work_of(a, blockIdx.z, blockIdx.y, 0, 0x3fffffff, &w)) return;
    const int tile = w.t0 + (int)blockIdx.x * kWaves + wave;
    if (tile >= w.t1) return;
    const uint8_t *p = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, w.b, w.h, tile);
    if (!p) return;
    const CodeConsts cc = code_consts<BF>();
    u4 kc[2][kSteps];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const u4 words = *reinterpret_cast<const u4 *>(p + 1024 * j + 16 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) kc[(4 * j + i) / kSteps][(4 * j + i) % kSteps] = codes16<BF>(words[i], cc);
    }
    const uint32_t *params = reinterpret_cast<const uint32_t *>(p + 2 * T::kCodes);
    for (int j = lane; j < 32 * NG; j += 64) shared[wave][j] = params[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    float st[NG][8], off[NG][8];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t v = shared[wave][32 * g + 16 * (e >> 2) + 4 * b4 + (e & 3)];
            st[g][e] = par_step<BF>(v);
            off[g][e] = par_offset<BF>(v);
        }
    const int G = a.q_heads / a.c.kv_heads, base = 32 * tile;
    const float c1 = a.scale * kLog2e;
    // rows that see any slot of the tile: with a causal mask those from the slots' own on
    const int i0 = a.causal ? max(0, base - (w.len - w.n)) : 0;
    const int i1 = a.window > 0 ? min(w.n, base + 31 + a.window - (w.len - w.n)) : w.n;
    float mass[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int row0 = i0 * G / 16 * 16; row0 < i1 * G; row0 += 16) {
        const int row = row0 + r;
        const bool there = row < w.rows;
        const int i = there ? row / G : 0;
        const int head = w.h * G + (there ? row - i * G : 0);
        const int lo = there ? row_lo(i, w.n, w.len, a.window) : 0;
        const int hi = there ? row_hi(i, w.n, w.len, a.causal) : 0;
        const int64_t token = w.first + i;
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + token * a.q_stride + (int64_t)head * D + 8 * b4;
        const float lse = a.lse[token * a.q_heads + head];
        const float shift = lse == -__builtin_inff() ? lse : -lse * kLog2e;     // (a row that saw nothing adds nothing)
        u4 q[kSteps];
        float qsum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) qsum[g] = 0.f;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            q[j] = *reinterpret_cast<const u4 *>(src + 32 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) qsum[j / kPer] += lo_f32<BF>(q[j][e]) + hi_f32<BF>(q[j][e]);
        }
        f4 init[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            qsum[g] += __shfl_xor(qsum[g], 16);
            qsum[g] += __shfl_xor(qsum[g], 32);
            const float z = -16.0f * qsum[g];
            init[g] = f4{z, z, z, z};
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            float x[4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f4 acc = init[g];
#pragma unroll
                for (int j = g * kPer; j < (g + 1) * kPer; ++j) acc = mfma16x16x32_t<BF>(kc[sub][j], q[j], acc);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = g == 0 ? off[0][4 * sub + e] * qsum[0] : __builtin_fmaf(off[g][4 * sub + e], qsum[g], x[e]);
                    x[e] = __builtin_fmaf(st[g][4 * sub + e], acc[e], x[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int slot = base + 16 * sub + 4 * b4 + e;
                const bool ok = slot >= lo && slot < hi;
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], c1, shift));
                mass[4 * sub + e] += ok ? y : 0.f;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int d = 1; d < 16; d *= 2) mass[e] += __shfl_xor(mass[e], d);
        const int slot = base + 16 * (e >> 2) + 4 * b4 + (e & 3);
        if (r == 0 && slot < w.len) {
            float *to = a.acc + ((int64_t)w.b * a.c.kv_heads + w.h) * a.acc_stride + slot;
            *to += mass[e];
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

size_t kv4_attention_workspace_bytes(const Kv4AttnArgs &a) {
    const Plan p = plan_of(a);
    if (p.chunks <= 1) return 0;
    return (size_t)a.c.batch * a.c.kv_heads * p.row_tiles * p.chunks * 16 * p.nt * (a.c.head_dim + 2) * 4;
}

hipError_t launch_kv4_attention(const Kv4AttnArgs &a, hipStream_t stream) {
    const Plan p = plan_of(a);
    const dim3 grid((unsigned)p.chunks, (unsigned)(a.c.kv_heads * p.row_tiles), (unsigned)a.c.batch);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        if (p.nt == 1)
            attend_kernel<bf(), d(), ng(), 1><<<grid, kThreads, 0, stream>>>(a, p);
        else if constexpr (d() <= 128)
            attend_kernel<bf(), d(), ng(), 2><<<grid, kThreads, 0, stream>>>(a, p);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && p.chunks > 1) {
            join_kernel<bf(), d()><<<dim3(16 * p.nt, grid.y, grid.z), d(), 0, stream>>>(a, p);
            e = hipGetLastError();
        }
        return e;
    });
}

hipError_t launch_kv4_mass(const Kv4AttnArgs &a, hipStream_t stream) {
    const int tiles = (a.max_kv + 31) / 32;
    const dim3 grid((unsigned)((tiles + kWaves - 1) / kWaves), (unsigned)a.c.kv_heads, (unsigned)a.c.batch);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        mass_kernel<bf(), d(), ng()><<<grid, kThreads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace w4a16
