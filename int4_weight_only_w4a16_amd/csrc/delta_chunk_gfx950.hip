// The gated delta rule for prompts, and for trees of drafted tokens, 64 tokens at a time.
//
// In a chunk with G_i the sum of g up to token i, from the state S at its start (K, Q, V its rows,
// each key and query of unit length if asked for):
//   A_ij = beta_i e^(G_i - G_j) k_i . k_j  (j < i),   T = (I + A)^-1 diag(beta)
//   U = T (V - e^G K S)                               the rows that the tokens write
//   O = scale (e^G Q S + [e^(G_i - G_j) q_i . k_j]_(j <= i) U)
//   S <- e^G_last S + (e^(G_last - G) K)^T U
// For a tree "j < i" is "i descends from j", G_i the sum along the path, and S stays.
//
// chunk_prep_kernel makes what does not depend on S, for all chunks at once: T, the triangle of
// products with the queries, and keys and queries as operands.  chunk_scan_kernel walks over the
// chunks of one head with sixteen columns of S in each wave (columns do not depend on each other):
// the state stays in the accumulators of the matrix instructions, and what one product leaves in
// a lane is the next one's operand as it stands, if the depth (channels, or tokens) is taken in
// the order slot 8 b + e = place 4 b + e of the first 16, 16 + 4 b + e - 4 of the next.  So waves
// exchange nothing.
//
// The state is fp32, and its sums keep that: each factor that is not an input enters in two
// 16-bit parts of eleven bits (S, the rows V - e^G K S, T, the rows e^(G_last - G) U), three
// products for a pair of such factors, lo x lo left out (2^-22).  Keys and queries of
// either type enter as they are, once a power of two for each row brings them into fp16's range, but for
// elements below about 2^-14 (keys; queries 2^-28) of their row's largest, which fp16's smallest place rounds: by at
// most 2^-25 (2^-39) of that largest.  So do powers of two for each row of T and each column of S and of the rows.
// What goes into the output alone has one part (2^-12), an eighth of a bfloat16 output's own rounding.  An fp16 output would be
// 1.7 times as far off as its rounding alone: there U has two parts and the triangle a second one
// of e4m3 (1.1 times; five prompts 112 -> 119 us); a tree's have two of S and U (1.2 times).
// Powers of two come off in fp32.
//
// Two parts hold 22 bits of what is within 2^-16 of the largest they are made with, and fewer of what is smaller:
// of a row of R beside a column's largest, which may be a later token's, or one that has faded by the chunk's end.
// So each chunk is looked at (least and weighed rows of R), and one where a row or the next state would lose by it
// is gone through token by token, in fp32 from the inputs (1.1 us a token; the look, and U's powers of two by its own
// largest, cost 3 to 5 %: 8191 tokens 297 -> 307 us, five prompts 120 -> 125).  So is a chunk with products that leave fp32.
//
// Bound by the chain of chunks: one sequence of 8191 tokens, 16 + 48 heads of 128 x 128, bfloat16,
// takes 76 us for the preparation and 242 to 256 for the scan, 1.9 a chunk (memory alone: 58).

// What is not finite (in a key, a gate, a value) would reach earlier rows, or a tree's other
// branches, through products with zero.  Its row is taken out as zeros and marked, and the rows
// that come after it, and S, become NaN.

#include <algorithm>
#include <type_traits>

#include "delta_device.hpp"
#include "lds.hpp"

namespace w4a16 {
namespace {

constexpr int kChunk = 64;
constexpr int kTop = 14;               // operands lie below 2^kTop
constexpr int kTopK = 0;               // and keys below 2^kTopK
constexpr int kTopU = 9;               // and rows of U for the next state below 2^kTopU
// What 16-bit parts take from a column's small rows for its largest's sake: from U as it comes out (rows of T below 2^14
// by rows of R below 2^14) about 2^-10, so that what an output adds up is to be kLeastU of those at least, kLost
// of R; from its weighed rows (2^-25 of U at most), the next state's, 2^-35, and kSmall of R in their heaviest.
constexpr float kLeastU = 2.0f, kLost = 1.0f / (1 << 26), kSmall = 1.0f / (1 << 17);
constexpr int kLeastWeighed = -15;
// Factors that chunks take: keys beside the longest, what comes off a row, products with queries, elements of T.  With rows and states below 2^100 none
// of what is made of them leaves fp32.
constexpr float kShortKey = 1.0f / (1 << 20), kMostRow = 1 << 24, kMostProduct = 0x1p32f, kMostT = 1 << 20;
constexpr int kWalked = -(1 << 30);    // in the place of U's power of two: the outputs are made already
constexpr float kRestUp = 64.f;        // what fp16 leaves of a number below 2^14 is at most 4; with this, 2^8
constexpr float kLog2e = 1.4426950408889634f;

// Workspace of one chunk: for each key head K and Q as operands (tiles of 1 KiB: 64 lanes x 16
// bytes; of K the first eight bytes of all lanes and then the others, so that its columns can be
// read without bank conflicts as well), for each value head T in two parts, the products with the queries (the six tiles of 16 x 32
// that are not above the diagonal), and what goes by rows.
// For fp16 also what those products leave of their rounding, in e4m3.
template <bool BF, int DK>
struct Chunk {
    static constexpr int kTiles = DK / 8;                      // of K and Q each
    static constexpr int kKey = 2 * kTiles * 1024;
    static constexpr int kHigh = 0, kLow = 6 * 1024, kWithin = 12 * 1024, kRest = 18 * 1024, kRows = BF ? kRest : 21 * 1024;
    static constexpr int kValue = kRows + 2 * 1024;
    // in kRows: fp32 [64] each: what comes off a row (e^G |k|-scale), what weighs a row of U for S, for the
    // output of S and of U; e^G_last, the power of two in the second of them; whether something is
    // beyond; what the last sixteen rows count for S, of the heaviest (NaN then); e^g, T's power of two, and its diagonal
    static constexpr int kOff = 0, kWeigh = 256, kFromS = 512, kFromU = 768, kLast = 1024, kHeavy = 1040, kKeep = 1280, kTau = 1536, kDiagonal = 1792;
};

// The part of a call that one launch works on: `chunks` chunks from the first_chunk-th of `batch`
// sequences from the first_seq-th.
struct Segment {
    int first_seq, batch, first_chunk, chunks;
    uint8_t *keys, *values;            // [batch][chunks][heads][bytes]
    float *carry;                      // [batch][v_heads][DK][value_dim]: states that are not in the pool
};

__device__ __forceinline__ int exponent(float v) { return __builtin_amdgcn_frexp_expf(v); }
__device__ __forceinline__ float times2(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }
__device__ __forceinline__ float exp_f32(float x) { return __builtin_amdgcn_exp2f(kLog2e * x); }
// Row (or column) r of what lane (r, b) holds as operand s: places 4 b .. of two tiles of 16.
__device__ __forceinline__ int place(int s, int b, int e) { return 32 * s + 16 * (e >> 2) + 4 * b + (e & 3); }

// First tile of row tile mt among those that are not above the diagonal.
__device__ __forceinline__ constexpr int tile_of(int mt, int s) { return mt < 2 ? mt : 2 * mt - 2 + s; }

// x by and y by rounded to fp16, and what that leaves, rounded too.  (The first parts are pinned: made
// twice, by instructions that round ties to different sides, they would not go with the second.)
__device__ __forceinline__ void split2(float x, float y, float by, uint32_t *hi, uint32_t *lo) {
    *hi = pack2<false>(x * by, y * by);
    asm("" : "+v"(*hi));
    *lo = pack2<false>(__builtin_fmaf(x, by, -lo_f32<false>(*hi)), __builtin_fmaf(y, by, -hi_f32<false>(*hi)));
}

// Two operands of eleven bits each from eight fp32 values times `by`.
struct Split {
    h8 hi, lo;
};
__device__ __forceinline__ Split split(const f4 &x, const f4 &y, float by) {
    u4 hi, lo;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t h, l;
        split2(x[2 * e], x[2 * e + 1], by, &h, &l);
        hi[e] = h;
        lo[e] = l;
        split2(y[2 * e], y[2 * e + 1], by, &h, &l);
        hi[2 + e] = h;
        lo[2 + e] = l;
    }
    return {__builtin_bit_cast(h8, hi), __builtin_bit_cast(h8, lo)};
}

// An operand of e4m3 from eight fp32 values times `by`.
__device__ __forceinline__ int64_t in_fp8(const f4 &x, const f4 &y, float by) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, 0, false);
    const int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * by, y[1] * by, 0, false);
    return __builtin_bit_cast(int64_t, u2{(uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true),
                                          (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2] * by, y[3] * by, hi, true)});
}

// The largest over the 16 lanes of a row of lanes (DPP: no LDS).
__device__ __forceinline__ float top_of_row(float v) {
#define W4A16_TOP_ROR(N) \
    v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + N, 0xF, 0xF, true)))
    W4A16_TOP_ROR(8);
    W4A16_TOP_ROR(4);
    W4A16_TOP_ROR(2);
    W4A16_TOP_ROR(1);
#undef W4A16_TOP_ROR
    return v;
}

// The largest size in a column's lanes; NaN if there is one.
__device__ __forceinline__ float top_of_column(float v) {
    const uint32_t bits = __float_as_uint(v);
    const auto halves = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
    const float w = __builtin_elementwise_maximum(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
    const uint32_t half = __float_as_uint(w);
    const auto rows = __builtin_amdgcn_permlane16_swap(half, half, false, false);
    return __builtin_elementwise_maximum(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
}

// One token of a head for the columns of a wave, in fp32 throughout: moves S on
// (rows 16 t + 4 b + j of column `col`, the (lane % 16)-th of the wave's) and returns the output.
template <bool BF, int DK>
__device__ __forceinline__ float one_token(const DeltaArgs &a, int64_t row, int h, int col, int b, float keep, float beta,
                                           f4 (&S)[DK / 16]) {
    constexpr int kTiles = DK / 16;
    const int hk = h / (a.v_heads / a.k_heads);
    const uint16_t *const qr = static_cast<const uint16_t *>(a.q) + row * a.q_stride + hk * DK + 4 * b;
    const uint16_t *const kr = static_cast<const uint16_t *>(a.k) + row * a.k_stride + hk * DK + 4 * b;
    const float v = lo_f32<BF>(static_cast<const uint16_t *>(a.v)[row * a.v_stride + (int64_t)h * a.value_dim + col]);
    float q[4 * kTiles], k[4 * kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const u2 q4 = *reinterpret_cast<const u2 *>(qr + 16 * t), k4 = *reinterpret_cast<const u2 *>(kr + 16 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            q[4 * t + 2 * i] = lo_f32<BF>(q4[i]);
            q[4 * t + 2 * i + 1] = hi_f32<BF>(q4[i]);
            k[4 * t + 2 * i] = lo_f32<BF>(k4[i]);
            k[4 * t + 2 * i + 1] = hi_f32<BF>(k4[i]);
        }
    }
    if (a.unit) {
        to_unit<16>(k, a.eps);
        to_unit<16>(q, a.eps);
    }
    // (the output from the new state, not by q . k, which may leave fp32)
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sk = __builtin_fmaf(S[t][j], k[4 * t + j], sk);
    const float u = beta * (v - keep * over_lanes<16>(sk));
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[t][j] = __builtin_fmaf(k[4 * t + j], u, keep * S[t][j]);
            sq = __builtin_fmaf(S[t][j], q[4 * t + j], sq);
        }
    return a.scale * over_lanes<16>(sq);
}

constexpr int kMostHeads = 4;          // value heads of a workgroup

// One chunk of `heads` value heads that share a key head: what the heads have in common, the products of
// keys with keys and queries among it, is made once.  TREE: of one head, and its outputs as well, since there
// is no next chunk (8 trees of 12 to 47 drafts, 48 heads: 25 us; with the outputs in a launch of their own once 36 to 23).
template <bool BF, int DK, bool TREE>
__global__ void __launch_bounds__(256, TREE ? 2 : 4) chunk_prep_kernel(DeltaArgs a, Segment seg, int heads) {
    using C = Chunk<BF, DK>;
    constexpr int kStride = DK + 8, kA = 68, kP = 72;
    // keys and queries, and A and X (of a chunk among others in their place)
    constexpr int kPart = kChunk * (2 * kStride > 4 * kA ? 2 * kStride : 4 * kA);
    __shared__ __align__(16) uint8_t shared[TREE ? 4 : 2][kPart];
    __shared__ __align__(16) float tree_rows[TREE ? 4 * kChunk : 4];
    auto &K = *reinterpret_cast<_Float16(*)[kChunk][kStride]>(shared[0]);
    auto &Q = *reinterpret_cast<_Float16(*)[kChunk][kStride]>(shared[1]);
    auto &A = *reinterpret_cast<float(*)[kChunk][kA]>(shared[TREE ? 2 : 0]);
    auto &X = *reinterpret_cast<float(*)[kChunk][kA]>(shared[TREE ? 3 : 1]);
    __shared__ double all_G[kMostHeads][kChunk];
    __shared__ __align__(16) float all_beta[kMostHeads][kChunk];
    __shared__ __align__(16) float kf[kChunk], qf[kChunk];
    __shared__ int tau[kChunk];
    __shared__ uint64_t kin[kChunk];
    __shared__ uint64_t redo_rows[TREE ? 16 : 1];      // of a group of columns, rows that go token by token
    __shared__ int marks[4];                   // of a wave: factors beyond what products of them hold
    __shared__ uint32_t bad_row[kChunk], bad_gate[kMostHeads][kChunk];     // 1: the key, 2: the query; a gate

    const int ci = blockIdx.x, h0 = blockIdx.y * heads, r = a.v_heads / a.k_heads, hk = h0 / r;
    Seq s;
    if (!seq_of(a.s, seg.first_seq + blockIdx.z, &s)) return;
    if (TREE) s.n = min(s.n, kChunk);
    const int t0 = kChunk * (seg.first_chunk + ci);
    if (t0 >= s.n) return;
    const int n = min(kChunk, s.n - t0);
    const int row_tiles = TREE ? (n + 15) / 16 : 4;        // of a tree those with tokens alone
    const int64_t slot = (int64_t)blockIdx.z * seg.chunks + ci;
    uint8_t *const to_key = seg.keys + (slot * a.k_heads + hk) * C::kKey;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), my_lane = tid & 63;
    int lane = my_lane, m = lane & 15, b = lane >> 4;

    // of a tree, the state: two groups of sixteen columns at a time in each wave
    constexpr int kRowTiles = DK / 16, kSteps = DK / 32;
    f4 S[TREE ? 2 : 1][kRowTiles];
    auto load_state = [&](int g0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int g = min(g0 + 4 * u, a.value_dim / 16 - 1);
            const float *const from = a.state + ((max(s.state, (int64_t)0) * a.v_heads + h0) * DK + 4 * b) * a.value_dim + 16 * g + m;
#pragma unroll
            for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[u][t][j] = s.fresh ? 0.f : from[(int64_t)(16 * t + j) * a.value_dim];
        }
    };
    u4 raw[2][DK / 32];                        // a quarter of a row of K and of Q
    const int my_row = tid >> 2, my_part = (tid & 3) * (DK / 4);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint16_t *const src = (which ? static_cast<const uint16_t *>(a.q) + (s.first + t0 + my_row) * a.q_stride
                                           : static_cast<const uint16_t *>(a.k) + (s.first + t0 + my_row) * a.k_stride) +
                                    hk * DK + my_part;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i)
            raw[which][i] = my_row < n ? *reinterpret_cast<const u4 *>(src + 8 * i) : u4{0u, 0u, 0u, 0u};
    }
    if constexpr (TREE) load_state(wave);

    // ---- gates, a head in each wave, and their sums in 64 bits: differences of far sums keep their precision ----
    uint64_t word = (2ull << lane) - 1;
    if constexpr (TREE) word = lane < n ? ((uint64_t)a.s.tree[s.first + lane] & ((1ull << lane) - 1)) | 1ull << lane : 0;
    if (wave == 0) kin[lane] = word;
    if (wave < heads) {
        const int h = h0 + wave;
        Gates gate{0.f, 0.f};
        if (lane < n)
            gate = gates_of<BF>(a, s.first + t0 + lane, h, a.a_log ? expf(a.a_log[h]) : 0.f, a.a_log ? a.dt_bias[h] : 0.f);
        const bool ok = gate.g < __builtin_inff() && __builtin_fabsf(gate.beta) < __builtin_inff();
        // (e^-256 is 0 in fp32, as is all that it multiplies)
        const double g = ok ? (double)fmaxf(gate.g, -256.f) : 0.0;
        double sum = g;
        if constexpr (TREE) {
            sum = 0;
            const uint64_t bits = __builtin_bit_cast(uint64_t, g);
            for (int j = 0; j < n; ++j) {
                const uint64_t of_j = (uint32_t)__builtin_amdgcn_readlane((uint32_t)bits, j) |
                                      (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(bits >> 32), j) << 32;
                sum += word >> j & 1 ? __builtin_bit_cast(double, of_j) : 0.0;
            }
        } else {
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double below = __shfl_up(sum, d);
                if (lane >= d) sum += below;
            }
        }
        all_beta[wave][lane] = ok ? gate.beta : 0.f;
        all_G[wave][lane] = sum;
        bad_gate[wave][lane] = ok ? 0u : 1u;
    }

    // ---- keys and queries as fp16 rows of a common size, and what came off them ----
    uint32_t bad = 0;
    bool large = false;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint32_t limit = BF ? 0x7F80u : 0x7C00u;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(raw[which][i][e] & 0x7FFFu, raw[which][i][e] >> 16 & 0x7FFFu));
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const bool fine = top < limit;
        const int up = fine && top ? min((which ? kTop : kTopK) - exponent(lo_f32<BF>(top)), 126) : 0;
        const float by = fine ? times2(1.0f, up) : 0.f;
        float sum = 0.f;
        _Float16 *const dst = (which ? Q[my_row] : K[my_row]) + my_part;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            h8 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = fine ? lo_f32<BF>(raw[which][i][e]) * by : 0.f;
                const float x1 = fine ? hi_f32<BF>(raw[which][i][e]) * by : 0.f;
                sum = __builtin_fmaf(x0, x0, sum);
                sum = __builtin_fmaf(x1, x1, sum);
                v[2 * e] = (_Float16)x0;
                v[2 * e + 1] = (_Float16)x1;
            }
            *reinterpret_cast<h8 *>(dst + 8 * i) = v;
        }
        sum += __shfl_xor(sum, 1);
        sum += __shfl_xor(sum, 2);
        if (my_part == 0) {
            // (rows past the sequence's are zeros and count for nothing)
            const float eps = times2(a.eps, 2 * up);       // (infinite: then it is all that there is)
            float f = !a.unit                  ? times2(1.0f, -up)
                      : eps < __builtin_inff() ? 1.0f / sqrtf(sum + eps)
                                               : times2(1.0f / sqrtf(a.eps), -up);
            // (nor does a row of zeros, with 1 / sqrt(eps))
            if (my_row >= n || (top == 0 && f < __builtin_inff())) f = 0.f;
            const bool ok = fine && f < __builtin_inff();
            large |= !(f * (which ? a.scale : 1.0f) < kMostRow);
            (which ? qf : kf)[my_row] = ok ? f : 0.f;
            if (!ok) bad |= 1u + which;
            if (which) bad_row[my_row] = bad;
        }
    }
    __syncthreads();

    if (wave == 0) {
        // (products with long keys would take the short ones' bits, though their tokens may write nothing)
        const float mine = kf[lane];
        large |= mine > 0.f && mine < top_of_column(top_of_row(mine)) * kShortKey;
    }

    // ---- keys and queries as operands ----
    if (!TREE && h0 % r == 0) {
#pragma unroll
        for (int i = 0; i < C::kTiles / 4; ++i) {
            const int tile = 4 * i + wave;                 // [row tile][DK / 32]
            const int row = 16 * (tile / (DK / 32)) + m, ch = 32 * (tile % (DK / 32)) + 4 * b;
            const h4 k0 = *reinterpret_cast<const h4 *>(&K[row][ch]), k1 = *reinterpret_cast<const h4 *>(&K[row][ch + 16]);
            const h4 q0 = *reinterpret_cast<const h4 *>(&Q[row][ch]), q1 = *reinterpret_cast<const h4 *>(&Q[row][ch + 16]);
            *reinterpret_cast<h4 *>(to_key + 1024 * tile + 8 * lane) = k0;
            *reinterpret_cast<h4 *>(to_key + 1024 * tile + 512 + 8 * lane) = k1;
            *reinterpret_cast<h8 *>(to_key + 1024 * (C::kTiles + tile) + 16 * lane) =
                __builtin_shufflevector(q0, q1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // ---- products of keys with keys and queries; lane (m, b): rows 16 wave + 4 b + j, column 16 nt + m ----
    f4 kk[4], qk[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) kk[nt] = qk[nt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < DK / 32; ++d) {
        const h8 ka = *reinterpret_cast<const h8 *>(&K[16 * wave + m][32 * d + 8 * b]);
        const h8 qa = *reinterpret_cast<const h8 *>(&Q[16 * wave + m][32 * d + 8 * b]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt > wave) continue;
            const h8 kb = *reinterpret_cast<const h8 *>(&K[16 * nt + m][32 * d + 8 * b]);
            kk[nt] = mfma16x16x32(ka, kb, kk[nt]);
            qk[nt] = mfma16x16x32(qa, kb, qk[nt]);
        }
    }
    {
        const f4 of_k = *reinterpret_cast<const f4 *>(&kf[16 * wave + 4 * b]), of_q = *reinterpret_cast<const f4 *>(&qf[16 * wave + 4 * b]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt > wave) continue;
            const int col = 16 * nt + m;
            const float kc = kf[col];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kk[nt][j] = col < 16 * wave + 4 * b + j ? of_k[j] * kk[nt][j] * kc : 0.f;
                qk[nt][j] = a.scale * (of_q[j] * qk[nt][j] * kc);
            }
        }
    }

    for (int hi = 0; hi < heads; ++hi) {
        // (opaque: else every address that they go into is kept in registers through the loop, 120 more than there are)
        asm volatile("" : "+v"(lane), "+v"(m), "+v"(b));
        const int h = h0 + hi;
        const double *const G = all_G[hi];
        const float *const beta = all_beta[hi];
        uint8_t *const to = seg.values + (slot * a.v_heads + h) * C::kValue;
        __syncthreads();                       // keys and queries, or the head before, are done with
        f4 p[4];
        bool beyond = large;
        {
            // (all that is read comes before A is written, which the compiler takes to overlap it)
            const int row0 = 16 * wave + 4 * b;
            double of_row[4], of_col[4];
            uint64_t words[TREE ? 4 : 1];
            f4 strength;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                of_row[j] = G[row0 + j];
                of_col[j] = G[16 * j + m];
                strength[j] = beta[row0 + j];
                if constexpr (TREE) words[j] = kin[row0 + j];
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                if (nt > wave) continue;
                const int col = 16 * nt + m;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool sees = TREE ? words[TREE ? j : 0] >> col & 1 : col <= row0 + j;
                    const float w = sees ? exp_f32((float)(of_row[j] - of_col[nt])) : 0.f;
                    // (selects: a product may be infinite)
                    A[row0 + j][col] = sees ? strength[j] * (kk[nt][j] * w) : 0.f;
                    p[nt][j] = sees ? qk[nt][j] * w : 0.f;
                    beyond |= !(__builtin_fabsf(p[nt][j]) < kMostProduct);
                }
            }
        }
        __syncthreads();

        // ---- X = (I + A)^-1: blocks of 16 on the diagonal by substitution, the others from them ----
        {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = i == m ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) v = __builtin_fmaf(-A[16 * wave + i][16 * wave + j], x[j], v);
                x[i] = v;
                if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);       // (else all of A's rows come into registers first)
            }
            f4 mine = {0.f, 0.f, 0.f, 0.f};    // rows 4 b + e of the block
#pragma unroll
            for (int i = 0; i < 16; ++i) mine[i & 3] = b == i / 4 ? x[i] : mine[i & 3];
#pragma unroll
            for (int e = 0; e < 4; ++e) X[16 * wave + 4 * b + e][16 * wave + m] = mine[e];
            __syncthreads();
            // a wave's column of blocks below: X_ij = -X_ii sum_(j <= k < i) A_ik X_kj, its own X_kj in registers as
            // the products leave them, which is how they go into the next
            f4 column[4];
            column[0] = mine;
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int i = wave + d;
                if (i >= row_tiles) break;
                f4 left[4], acc = {0.f, 0.f, 0.f, 0.f}, out = acc;
#pragma unroll
                for (int k = 0; k < d; ++k) left[k] = *reinterpret_cast<const f4 *>(&A[16 * i + m][16 * (wave + k) + 4 * b]);
                left[3] = *reinterpret_cast<const f4 *>(&X[16 * i + m][16 * i + 4 * b]);
#pragma unroll
                for (int k = 0; k < d; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(left[k][e], column[k][e], acc, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) out = __builtin_amdgcn_mfma_f32_16x16x4f32(left[3][e], acc[e], out, 0, 0, 0);
                column[d] = -out;
#pragma unroll
                for (int e = 0; e < 4; ++e) X[16 * i + 4 * b + e][16 * wave + m] = column[d][e];
            }
        }
        __syncthreads();

        // ---- T = X diag(beta) as operands; lane (m, b): row 16 wave + m ----
        {
            const int row = 16 * wave + m;
            float t[2][8], top = 0.f;
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const int col = place(d, b, e);
                    const bool in = 2 * d + (e >> 2) <= wave;
                    f4 v = {0.f, 0.f, 0.f, 0.f}, w = v;
                    if (in) {
                        v = *reinterpret_cast<const f4 *>(&X[row][col]);
                        w = *reinterpret_cast<const f4 *>(&beta[col]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        t[d][e + i] = v[i] * w[i];
                        top = __builtin_elementwise_maximum(top, __builtin_fabsf(t[d][e + i]));
                    }
                }
            beyond |= !(top < kMostT) && row < n;
            const int up = kTop - max(exponent(top_of_column(top)), -60);
            if (b == 0) tau[row] = up;
            if (__builtin_amdgcn_ballot_w64(beyond) == 0) {
                if (lane == 0) marks[wave] = 0;
            } else if (lane == 0) {
                marks[wave] = 1;
            }
            if constexpr (TREE) __syncthreads();               // X is done with: T comes in its place
            uint8_t *const tiles = TREE ? reinterpret_cast<uint8_t *>(&X[0][0]) : to;
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                if (2 * d > wave) continue;
                const Split x = split(f4{t[d][0], t[d][1], t[d][2], t[d][3]}, f4{t[d][4], t[d][5], t[d][6], t[d][7]}, times2(1.0f, up));
                const int tile = tile_of(wave, d);
                *reinterpret_cast<h8 *>(tiles + C::kHigh + 1024 * tile + 16 * lane) = x.hi;
                *reinterpret_cast<h8 *>(tiles + C::kLow + 1024 * tile + 16 * lane) = x.lo;
            }
        }
        __syncthreads();

        // ---- products with the queries: by what the rows of U carry, through LDS into operands ----
        _Float16 *const P = reinterpret_cast<_Float16 *>(&A[0][0]);      // [64][kP]
        uint8_t *const left = reinterpret_cast<uint8_t *>(P + kChunk * kP);
        static_assert(sizeof(A) >= kChunk * kP * 3, "both in A's place");
        float *const rows = TREE ? tree_rows : reinterpret_cast<float *>(to + C::kRows);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt > wave) continue;
            // (what meets no row of U does not count for the power of two)
            const float down = beta[16 * nt + m] != 0.f ? times2(1.0f, -tau[16 * nt + m]) : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[nt][j] *= down;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * wave + 4 * b + j;
            float top = 0.f;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
                if (nt <= wave) top = fmaxf(top, __builtin_fabsf(p[nt][j]));
            const int up = kTop - max(exponent(top_of_row(top)), -100);
            const float by = times2(1.0f, up);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                uint32_t one = nt > wave ? 0 : pack2<false>(p[nt][j] * by, 0.f);
                asm("" : "+v"(one));           // (as in split2)
                P[row * kP + 16 * nt + m] = __builtin_bit_cast(h2, one)[0];
                if constexpr (!TREE && !BF) {
                    const float rest = nt > wave ? 0.f : __builtin_fmaf(p[nt][j], by, -lo_f32<false>(one)) * kRestUp;
                    left[row * kP + 16 * nt + m] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(rest, rest, 0, false);
                }
            }
            if (m == 0) rows[C::kFromU / 4 + row] = times2(1.0f, -up);
        }
        // (a wave reads the rows that it wrote)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            if (TREE || 2 * d > wave) continue;
            const _Float16 *const from = P + (16 * wave + m) * kP + 32 * d + 4 * b;
            const h4 lo = *reinterpret_cast<const h4 *>(from), hi4 = *reinterpret_cast<const h4 *>(from + 16);
            *reinterpret_cast<h8 *>(to + C::kWithin + 1024 * tile_of(wave, d) + 16 * lane) =
                __builtin_shufflevector(lo, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
            if constexpr (!BF) {
                const uint8_t *const rest = left + (16 * wave + m) * kP + 32 * d + 4 * b;
                *reinterpret_cast<u2 *>(to + C::kRest + 512 * tile_of(wave, d) + 8 * lane) =
                    u2{*reinterpret_cast<const uint32_t *>(rest), *reinterpret_cast<const uint32_t *>(rest + 16)};
            }
        }

        // ---- what goes by rows ----
        if (wave == 0) {
            const float grow = exp_f32((float)G[lane]), nan = __builtin_nanf("");
            const float weigh = times2(exp_f32((float)(G[kChunk - 1] - G[lane])) * kf[lane], -tau[lane]);
            const int up = -25 - max(exponent(top_of_column(top_of_row(weigh))), -120);
            rows[C::kOff / 4 + lane] = (bad_row[lane] & 1) | bad_gate[hi][lane] ? nan : grow * kf[lane];
            // (of a tree, T's diagonal, infinite where nothing is written)
            const float diagonal = times2(__builtin_fabsf(beta[lane]), tau[lane]);
            if (TREE) rows[C::kWeigh / 4 + lane] = diagonal == 0.f || lane >= n ? __builtin_inff() : diagonal;
            else rows[C::kWeigh / 4 + lane] = times2(weigh, up);
            rows[C::kFromS / 4 + lane] = bad_row[lane] & 2 ? nan : a.scale * qf[lane] * grow;
            if constexpr (!TREE) {
                rows[C::kKeep / 4 + lane] = exp_f32((float)(G[lane] - (lane ? G[lane - 1] : 0.0)));
                reinterpret_cast<int *>(rows)[C::kTau / 4 + lane] = tau[lane];
                rows[C::kDiagonal / 4 + lane] = diagonal;
                const float counts = times2(__builtin_fabsf(weigh * beta[lane]), tau[lane]);
                const float most = top_of_column(top_of_row(counts));
                const int mark = marks[0] | marks[1] | marks[2] | marks[3];
                if (lane >= 48) rows[C::kHeavy / 4 + lane - 48] = mark ? nan : most > 0.f ? counts / most : 1.f;
                if (lane == 0) reinterpret_cast<int *>(rows)[C::kLast / 4 + 2] = mark;
            }
            if (!TREE && lane == 0) {
                rows[C::kLast / 4] = exp_f32((float)G[kChunk - 1]);
                reinterpret_cast<int *>(rows)[C::kLast / 4 + 1] = up;
            }
        }
    }

    // ======== a tree's outputs: as chunk_scan_kernel has them, two groups of columns at a time ========
    if constexpr (TREE) {
        __syncthreads();
        const bool marked = __builtin_amdgcn_readfirstlane(marks[0] | marks[1] | marks[2] | marks[3]) != 0;
        const uint8_t *const tiles = reinterpret_cast<const uint8_t *>(&X[0][0]);
        const _Float16 *const P = reinterpret_cast<const _Float16 *>(&A[0][0]);
        const int v_row = 2 * (int)a.v_stride, out_row = 2 * (int)a.out_stride;
        const auto from = make_rsrc(static_cast<const uint16_t *>(a.v) + s.first * a.v_stride, (uint32_t)(n * v_row));
        const auto into = make_rsrc(static_cast<const uint16_t *>(a.out) + s.first * a.out_stride, (uint32_t)(n * out_row));
        for (int g0 = wave; g0 < a.value_dim / 16; g0 += 8) {
            // (opaque: what does not change from one pair of groups to the next is not all kept in registers)
            asm volatile("" : "+v"(lane), "+v"(m), "+v"(b) : : "memory");
            if (g0 != wave) load_state(g0);
            int at[2];                         // bytes to this lane's column
#pragma unroll
            for (int u = 0; u < 2; ++u) at[u] = 2 * (h0 * a.value_dim + 16 * min(g0 + 4 * u, a.value_dim / 16 - 1) + m);
            uint16_t V[2][4][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        V[u][t][j] = __builtin_amdgcn_raw_buffer_load_b16(from, (16 * t + 4 * b + j) * v_row + at[u], 0, 0);
            Split x[2][kSteps];
            float of_s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float top = 0.f;
#pragma unroll
                for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_fabsf(S[u][t][j]));
                const int power = kTop - max(exponent(top_of_column(top)), -100);
                of_s[u] = times2(1.0f, -power);
#pragma unroll
                for (int d = 0; d < kSteps; ++d) x[u][d] = split(S[u][2 * d], S[u][2 * d + 1], times2(1.0f, power));
            }
            f4 ks[2][4], qs[2][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) ks[0][t] = ks[1][t] = qs[0][t] = qs[1][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t >= row_tiles) break;
#pragma unroll
                for (int d = 0; d < kSteps; ++d) {
                    const _Float16 *const kr = &K[16 * t + m][32 * d + 4 * b], *const qr = &Q[16 * t + m][32 * d + 4 * b];
                    const h8 k = __builtin_shufflevector(*reinterpret_cast<const h4 *>(kr), *reinterpret_cast<const h4 *>(kr + 16), 0, 1, 2, 3, 4, 5, 6, 7);
                    const h8 q = __builtin_shufflevector(*reinterpret_cast<const h4 *>(qr), *reinterpret_cast<const h4 *>(qr + 16), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        ks[u][t] = mfma16x16x32(k, x[u][d].hi, ks[u][t]);
                        qs[u][t] = mfma16x16x32(q, x[u][d].hi, qs[u][t]);
                        ks[u][t] = mfma16x16x32(k, x[u][d].lo, ks[u][t]);
                        qs[u][t] = mfma16x16x32(q, x[u][d].lo, qs[u][t]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (g0 + 4 * u >= a.value_dim / 16) break;
                f4 R[4];
                float top = 0.f, least = __builtin_inff();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const f4 off = *reinterpret_cast<const f4 *>(&tree_rows[C::kOff / 4 + 16 * t + 4 * b]);
                    const f4 diagonal = *reinterpret_cast<const f4 *>(&tree_rows[C::kWeigh / 4 + 16 * t + 4 * b]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        R[t][j] = __builtin_fmaf(-(off[j] * of_s[u]), ks[u][t][j], lo_f32<BF>(V[u][t][j]));
                        top = __builtin_elementwise_maximum(top, __builtin_fabsf(R[t][j]));
                        least = fminf(least, __builtin_fabsf(R[t][j] * diagonal[j]));      // (0 x infinity does not count)
                    }
                }
                top = top_of_column(top);
                uint64_t lost = 0;             // rows that come after one that is not finite
                if (__builtin_amdgcn_ballot_w64(!(top < __builtin_inff()))) {
                    uint64_t found = 0;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            found |= __builtin_fabsf(R[t][j]) < __builtin_inff() ? 0ull : 1ull << (16 * t + 4 * b + j);
                    found |= __shfl_xor(found, 16);
                    found |= __shfl_xor(found, 32);
                    for (int row = 0; row < kChunk; ++row) lost |= kin[row] & found ? 1ull << row : 0ull;
                    top = 0.f;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            R[t][j] = lost >> (16 * t + 4 * b + j) & 1 ? 0.f : R[t][j];
                            top = fmaxf(top, __builtin_fabsf(R[t][j]));
                        }
                    top = top_of_column(top);
                }
                const int up = kTop - max(exponent(top), -100);
                // Rows of R that are lost beside larger ones of their column, another branch's perhaps: as in the
                // scan, but without the row before: what a row alone has by chance goes token by token too (one of some
                // 2^25 elements, bfloat16; fp16 outputs, rounded to eight times less, leave less to lose).
                const float small = times2(BF ? kLeastU / 2 : kLeastU, -up);
                uint64_t redo = 0;
                const bool beyond = top >= 0x1p100f || (top < 0x1p-100f && top > 0.f) || of_s[u] > 0x1p86f;
                if (marked || __builtin_amdgcn_ballot_w64(beyond || (least < small && top > 0.f))) {
                    uint64_t mine = marked || (beyond && top > 0.f) ? ~0ull : 0ull;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const f4 diagonal = *reinterpret_cast<const f4 *>(&tree_rows[C::kWeigh / 4 + 16 * t + 4 * b]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (__builtin_fabsf(R[t][j] * diagonal[j]) < small && top > 0.f)
                                mine |= 1ull << (16 * t + 4 * b + j);
                    }
                    if (!marked) mine &= ~lost;
#pragma unroll
                    for (int d = 1; d < 64; d *= 2) mine |= __shfl_xor(mine, d);
                    // and what descends from them, which may have nothing of its own
                    mine = __builtin_amdgcn_ballot_w64(lane < n && (kin[lane] & mine) != 0);
                    redo = mine;
                }
                redo_rows[g0 + 4 * u] = redo;
                const Split r0 = split(R[0], R[1], times2(1.0f, up)), r1 = split(R[2], R[3], times2(1.0f, up));
                f4 U[4], o[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) U[t] = o[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t >= row_tiles) break;
#pragma unroll
                    for (int d = 0; d <= t / 2; ++d) {
                        const h8 hi = *reinterpret_cast<const h8 *>(tiles + C::kHigh + 1024 * tile_of(t, d) + 16 * lane);
                        const h8 lo = *reinterpret_cast<const h8 *>(tiles + C::kLow + 1024 * tile_of(t, d) + 16 * lane);
                        const Split &rows = d ? r1 : r0;
                        U[t] = mfma16x16x32(hi, rows.hi, U[t]);
                        U[t] = mfma16x16x32(hi, rows.lo, U[t]);
                        U[t] = mfma16x16x32(lo, rows.hi, U[t]);
                    }
                }
                float top_u = 0.f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top_u = fmaxf(top_u, __builtin_fabsf(U[t][j]));
                const int up_u = kTop - max(exponent(top_of_column(top_u)), -60);
                const Split v[2] = {split(U[0], U[1], times2(1.0f, up_u)), split(U[2], U[3], times2(1.0f, up_u))};
                const float of_u = times2(1.0f, -up - up_u);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t >= row_tiles) break;
#pragma unroll
                    for (int d = 0; d <= t / 2; ++d) {
                        const _Float16 *const pr = P + (16 * t + m) * kP + 32 * d + 4 * b;
                        const h8 p = __builtin_shufflevector(*reinterpret_cast<const h4 *>(pr), *reinterpret_cast<const h4 *>(pr + 16), 0, 1, 2, 3, 4, 5, 6, 7);
                        o[t] = mfma16x16x32(p, v[d].hi, o[t]);
                        o[t] = mfma16x16x32(p, v[d].lo, o[t]);
                    }
                    const f4 fs = *reinterpret_cast<const f4 *>(&tree_rows[C::kFromS / 4 + 16 * t + 4 * b]);
                    const f4 fu = *reinterpret_cast<const f4 *>(&tree_rows[C::kFromU / 4 + 16 * t + 4 * b]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = 16 * t + 4 * b + j;
                        float y = __builtin_fmaf(fs[j] * of_s[u], qs[u][t][j], (fu[j] * of_u) * o[t][j]);
                        y = lost >> row & 1 ? __builtin_nanf("") : y;
                        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack2<BF>(y, 0.f), into, row * out_row + at[u], 0, 0);
                    }
                }
            }
        }

        // Those rows, a group of columns at a time: a row's state from the pool's, through the tokens that it descends from,
        // or on from the last row's where that is one of them.
#pragma unroll 1
        for (int g = wave; g < a.value_dim / 16; g += 4) {
            const uint64_t rows = redo_rows[g];
            uint64_t todo = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(rows >> 32)) << 32 |
                            (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)rows);
            if (todo == 0) continue;
            wait_loads<0>();                   // (these rows' stores above are done)
            asm volatile("" : "+v"(lane), "+v"(m), "+v"(b) : : "memory");
            const int col = 16 * g + m;
            Gates gate{0.f, 0.f};
            if (lane < n)
                gate = gates_of<BF>(a, s.first + lane, h0, a.a_log ? expf(a.a_log[h0]) : 0.f, a.a_log ? a.dt_bias[h0] : 0.f);
            const float all_keep = expf(gate.g);
            f4 from_there[kRowTiles];
            uint64_t seen = 0;                 // what that state has been through
#pragma unroll 1
            for (; todo; todo &= todo - 1) {
                const int row = __builtin_ctzll(todo);
                const uint64_t word = kin[row];
                const uint64_t path = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(word >> 32)) << 32 |
                                      (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)word);
                if (seen == 0 || (seen & ~path)) {
                    seen = 0;
                    const float *const from = a.state + ((max(s.state, (int64_t)0) * a.v_heads + h0) * DK + 4 * b) * a.value_dim + col;
#pragma unroll
                    for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) from_there[t][j] = s.fresh ? 0.f : from[(int64_t)(16 * t + j) * a.value_dim];
                }
                float o = 0.f;
#pragma unroll 1
                for (uint64_t left = path & ~seen; left; left &= left - 1) {
                    const int i = __builtin_ctzll(left);
                    const float keep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all_keep), i));
                    const float strength = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate.beta), i));
                    o = one_token<BF, DK>(a, s.first + i, h0, col, b, keep, strength, from_there);
                }
                seen = path;
                if (b == 0)
                    static_cast<uint16_t *>(a.out)[(s.first + row) * a.out_stride + (int64_t)h0 * a.value_dim + col] =
                        (uint16_t)pack2<BF>(o, 0.f);
            }
        }
    }
}

// Four rows of one column of an LDS tile [rows][16 WAVES columns] of 16-bit values: lane (m, b) hands in the
// place of row m / 4, columns 4 (m % 4) .. of its group's block and gets column m of all four.
typedef short s4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u2 read_column(const lds_u8 *p) {
    typedef __attribute__((address_space(3))) s4 lds_s4;
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)const_cast<lds_u8 *>(p)));
}

// A workgroup walks over the chunks with 16 GROUPS columns of one head.  Wave w < GROUPS takes what the
// next state needs, for sixteen columns; wave GROUPS + w (with four groups on the same SIMD) their outputs, from the state and
// the rows U that the first hands over in LDS, and the copies.  (All in one wave, the only one on its SIMD,
// a chunk took 9300 cycles, of which instructions took 3300; now about 4500.)
template <bool BF, int DK, int GROUPS>
__global__ void __launch_bounds__(128 * GROUPS) chunk_scan_kernel(DeltaArgs a, Segment seg) {
    using C = Chunk<BF, DK>;
    constexpr int kSteps = DK / 32, kRowTiles = DK / 16;
    // two chunks, each with V's columns of this workgroup; and for each group the state as operands, U, what
    // comes off their sums, and rows that are lost
    constexpr int kColumnBytes = 32 * GROUPS, kTile = kChunk * kColumnBytes, kStage = C::kKey + C::kValue + kTile;
    constexpr int kU = kSteps * 1024, kFactors = kU + 4096, kHand = kFactors + 256;
    __shared__ __align__(16) uint8_t lds_raw[2 * kStage + GROUPS * kHand];
    lds_u8 *const lds = (lds_u8 *)lds_raw;

    const int h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
    Seq s;
    if (!seq_of(a.s, seg.first_seq + blockIdx.z, &s)) return;
    const int first = kChunk * seg.first_chunk;
    if (first >= s.n) return;
    const int count = min(seg.chunks, (s.n - first + kChunk - 1) / kChunk);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = wave % GROUPS;
    const int lane = threadIdx.x & 63, m = lane & 15, b = lane >> 4;
    const int col = 16 * (blockIdx.x * GROUPS + group) + m;
    lds_u8 *const hand = lds + 2 * kStage + group * kHand;

    if (wave >= GROUPS) {
        // ======== outputs and copies ========
        const lds_u8 *const factors = hand + kFactors + 4 * m, *const lost_at = hand + kFactors + 128 + 8 * m;
        const int64_t slot = (int64_t)blockIdx.z * seg.chunks;
        // rows of V and of the output by offsets from a chunk's first (the host keeps strides below 2^23 elements)
        constexpr int kUnits = kColumnBytes / 16;          // 16-byte units of a row
        const int v_row = 2 * (int)a.v_stride, out_row = 2 * (int)a.out_stride;
        const int v_at = lane / kUnits * v_row + 16 * (lane % kUnits);
        auto copy = [&](int ci) {
            const uint8_t *const key = seg.keys + ((slot + ci) * a.k_heads + hk) * C::kKey;
            const uint8_t *const value = seg.values + ((slot + ci) * a.v_heads + h) * C::kValue;
            lds_u8 *const to = lds + (ci & 1) * kStage;
            static_assert(C::kKey / 1024 % GROUPS == 0, "the same in every wave");
#pragma unroll
            for (int u = 0; u < C::kKey; u += 1024 * GROUPS)
                copy_kib(key, C::kKey, u + 1024 * group, to + u + 1024 * group, lane);
#pragma unroll
            for (int u = 0; u < C::kValue; u += 1024 * GROUPS)
                if (u + 1024 * GROUPS <= C::kValue || u + 1024 * group < C::kValue)
                    copy_kib(value, C::kValue, u + 1024 * group, to + C::kKey + u + 1024 * group, lane);
            // rows past the sequence's come as zeros
            const int n = min(kChunk, s.n - first - kChunk * ci);
            const auto rsrc = make_rsrc(static_cast<const uint16_t *>(a.v) + (s.first + first + (int64_t)kChunk * ci) * a.v_stride +
                                            h * a.value_dim + blockIdx.x * (16 * GROUPS),
                                        (uint32_t)((n - 1) * v_row + kColumnBytes));
#pragma unroll
            for (int i = 0; i < kTile / 1024 / GROUPS; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + C::kKey + C::kValue + 1024 * (GROUPS * i + group)), 16,
                                                         v_at + (GROUPS * i + group) * (1024 / kColumnBytes) * v_row, 0, 0, 0);
        };
        // Outputs of a chunk are stored while the next one's U is made: between (1) and (2) this wave has time
        // left, between (2) and (1) the other one.  Through LDS (the state's place, once it is in
        // registers), so that a lane stores eight columns of a row.
        u2 made[4];
        bool walked = false;                   // they are there already: nothing is stored
        auto store = [&](int ci) {
            asm volatile("" ::: "memory");
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lds_u8 *const to = hand + 32 * (16 * t + 4 * b + 2 * j) + 2 * m;
                    lds_put(to, (uint16_t)made[t][j]);
                    lds_put(to + 32, (uint16_t)(made[t][j] >> 16));
                }
            asm volatile("" ::: "memory");
            const int n = min(kChunk, s.n - first - kChunk * ci);
            const auto rsrc = make_rsrc(static_cast<const uint16_t *>(a.out) + (s.first + first + (int64_t)kChunk * ci) * a.out_stride +
                                            h * a.value_dim + blockIdx.x * (16 * GROUPS) + 16 * group,
                                        walked ? 0u : (uint32_t)((n - 1) * out_row + 32));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 32 * i + (lane >> 1);
                const u4 eight = lds_get<u4>(hand + 32 * row + 16 * (lane & 1));
                __builtin_amdgcn_raw_buffer_store_b128(eight, rsrc, row * out_row + 16 * (lane & 1), 0, 0);
            }
        };
        // What the outputs of a chunk are made of waits in registers while the next one's copies are issued.
        f4 qs[4], fs[4], fu[4], U[4];
        h8 within[6];
        int64_t rest[BF ? 1 : 6];
        float of_s;
        int up_r;
        uint64_t lost;
        auto make = [&] {
            f4 o[4], r[4];
            // (by its own largest, not by the most that it may be, which would leave small rows fewer bits)
            float top = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_fabsf(U[t][j]));
            const int up_u = kTop - max(exponent(top_of_column(top)), -60);
            const float by = times2(1.0f, up_u), of_u = times2(1.0f, -up_u - up_r);
#pragma unroll
            for (int t = 0; t < 4; ++t) o[t] = r[t] = f4{0.f, 0.f, 0.f, 0.f};
            if constexpr (BF) {
                h8 u[2];
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[d][e] = (_Float16)(U[2 * d + (e >> 2)][e & 3] * by);
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int t = 2 * d; t < 4; ++t) o[t] = mfma16x16x32(within[tile_of(t, d)], u[d], o[t]);
            } else {
                const Split u[2] = {split(U[0], U[1], by), split(U[2], U[3], by)};
                const float by8 = by / kRestUp;
                const int64_t few[2] = {in_fp8(U[0], U[1], by8), in_fp8(U[2], U[3], by8)};
                // (these with accumulators of their own, and first: a product of one type does not wait for one of
                // another as long as it must, if it adds to it)
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int t = 2 * d; t < 4; ++t)
                        r[t] = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(rest[tile_of(t, d)], few[d], r[t], 0, 0, 0);
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int t = 2 * d; t < 4; ++t) o[t] = mfma16x16x32(within[tile_of(t, d)], u[d].hi, o[t]);
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int t = 2 * d; t < 4; ++t) o[t] = mfma16x16x32(within[tile_of(t, d)], u[d].lo, o[t]);
            }
            f4 y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[t][j] = __builtin_fmaf(fs[t][j] * of_s, qs[t][j], (fu[t][j] * of_u) * (BF ? o[t][j] : o[t][j] + r[t][j]));
            walked = false;
            if (__builtin_amdgcn_ballot_w64(lost != 0)) {
                walked = __builtin_amdgcn_readfirstlane(up_r) == kWalked;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[t][j] = lost >> (16 * t + 4 * b + j) & 1 ? __builtin_nanf("") : y[t][j];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) made[t] = pack4<BF>(y[t][0], y[t][1], y[t][2], y[t][3]);
        };
        copy(0);
        if (count > 1) copy(1);
        wait_loads<0>();
        lds_barrier();                         // (0) the first chunk is there
        for (int ci = 0; ci < count; ++ci) {
            const lds_u8 *const at = lds + (ci & 1) * kStage;
            const lds_u8 *const mine = at + 16 * lane, *const val = at + C::kKey, *const rows = val + C::kRows + 16 * b;
            lds_barrier();                     // (1) the state is handed over
            h8 x[kSteps], q[kSteps][4];
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
                x[d] = lds_get<h8>(hand + 1024 * d + 16 * lane);
#pragma unroll
                for (int t = 0; t < 4; ++t) q[d][t] = lds_get<h8>(mine + 1024 * (C::kTiles + t * kSteps + d));
            }
            if (ci > 0) make();
#pragma unroll
            for (int t = 0; t < 4; ++t) qs[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < kSteps; ++d)
#pragma unroll
                for (int t = 0; t < 4; ++t) qs[t] = mfma16x16x32(q[d][t], x[d], qs[t]);
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                within[i] = lds_get<h8>(val + C::kWithin + 1024 * i + 16 * lane);
                if constexpr (!BF) rest[i] = lds_get<int64_t>(val + C::kRest + 512 * i + 8 * lane);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                fs[t] = lds_get<f4>(rows + C::kFromS + 64 * t);
                fu[t] = lds_get<f4>(rows + C::kFromU + 64 * t);
            }
            if (ci > 0) store(ci - 1);
            // the next chunk is there; the two stores may be under way
            if (ci == 0) wait_loads<0>();
            else wait_loads<2>();
            lds_barrier();                     // (2) U is handed over, and all of this chunk's is in registers
            if (ci + 2 < count) copy(ci + 2);
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = lds_get<f4>(hand + kU + 1024 * t + 16 * lane);
            of_s = lds_get<float>(factors);
            up_r = lds_get<int>(factors + 64);
            lost = lds_get<uint64_t>(lost_at);
        }
        make();
        store(count - 1);
        wait_loads<0>();
        return;
    }

    // ======== the state: S 2^power, below 2^16; lane (m, b): rows 16 t + 4 b + j of its column ========
    f4 S[kRowTiles];
    int power;
    float *const pool = s.state < 0 ? seg.carry + ((int64_t)blockIdx.z * a.v_heads + h) * DK * a.value_dim
                                    : a.state + (s.state * a.v_heads + h) * DK * a.value_dim;
    {
        const bool zero = seg.first_chunk == 0 && s.fresh;
        const float *const from = pool + (int64_t)(4 * b) * a.value_dim + col;
        float top = 0.f;
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t][j] = zero ? 0.f : from[(int64_t)(16 * t + j) * a.value_dim];
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_fabsf(S[t][j]));
        power = kTop - max(exponent(top_of_column(top)), -100);
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t][j] = times2(S[t][j], power);
    }

    // Whether rows of R are lost beside larger ones of their column: of some output, all that it adds up is
    // small, its own row and the one before as far as it is kept (of a row alone, that is chance and no
    // loss); or all that the next state consists of, `of_old` of it the last one.  A row that is zero is
    // right, unless earlier ones fade: what it takes back of them is not.
    auto lose = [&](const f4 (&R)[4], float by, const lds_u8 *rows, float gamma, float of_old, int n, int lane, int b) {
        const float none = gamma < kSmall ? -1.f : 0.f;
        float top = 0.f, before = 0.f;
        bool is = false;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f4 keep = lds_get<f4>(rows + C::kKeep + 64 * t), weigh = lds_get<f4>(rows + C::kWeigh + 64 * t);
            const f4 diagonal = lds_get<f4>(rows + C::kDiagonal + 64 * t);
            const u4 tau = lds_get<u4>(rows + C::kTau + 64 * t);
            float u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __builtin_fabsf(diagonal[j] * (R[t][j] * by));
            // the row before the first of these four, without its power of two
            const float end = times2(u[3], -(int)tau[3]), below = __shfl(end, lane - 16);
            float back = b > 0 ? below : before;
            before = __shfl(end, lane + 48);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                is |= 16 * t + 4 * b + j < n && diagonal[j] != 0.f && __builtin_fabsf(R[t][j]) > none &&
                      __builtin_fmaf(keep[j], times2(back, (int)tau[j]), u[j]) < kLeastU;
                top = fmaxf(top, u[j] * weigh[j]);
                back = times2(u[j], -(int)tau[j]);
            }
        }
        top = fmaxf(top_of_column(top), of_old);
        return is || (top > 0.f && exponent(top) < kLeastWeighed);
    };

    // A chunk whose numbers the products' parts cannot hold beside each other, token by token from the inputs.
    auto walk = [&](int ci) {
        int n = min(kChunk, s.n - first - kChunk * ci), head = h, my_col = col, my_b = b;
        asm volatile("" : "+s"(n), "+s"(head), "+v"(my_col), "+v"(my_b));      // (nothing of this is made before the loop)
        const int64_t row0 = s.first + first + (int64_t)kChunk * ci;
        Gates gate{0.f, 0.f};                  // of 64 tokens, one in each lane
        if (lane < n) gate = gates_of<BF>(a, row0 + lane, head, a.a_log ? expf(a.a_log[head]) : 0.f,
                                          a.a_log ? a.dt_bias[head] : 0.f);
        const float all_keep = expf(gate.g);
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t][j] = times2(S[t][j], -power);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const float keep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all_keep), i));
            const float beta = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate.beta), i));
            const float o = one_token<BF, DK>(a, row0 + i, head, my_col, my_b, keep, beta, S);
            if (my_b == 0)
                static_cast<uint16_t *>(a.out)[(row0 + i) * a.out_stride + (int64_t)head * a.value_dim + my_col] =
                    (uint16_t)pack2<BF>(o, 0.f);
        }
        float top = 0.f;
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_fabsf(S[t][j]));
        power = kTop - max(exponent(top_of_column(top)), -100);
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[t][j] = times2(S[t][j], power);
    };

    // One chunk.  Without WARY, false if anything in it asks for a look: nothing is changed then, and the wary form
    // begins again (`again`: between the barriers (1) and (2)).
    auto one_chunk = [&](auto wary, int ci, bool again) __attribute__((always_inline)) {
        constexpr bool WARY = wary();
        const int lane = threadIdx.x & 63, m = lane & 15, b = lane >> 4;
        lds_u8 *const factors = hand + kFactors + 4 * m, *const lost_at = hand + kFactors + 128 + 8 * m;
        const lds_u8 *const at = lds + (ci & 1) * kStage, *const val = at + C::kKey;
        const lds_u8 *const rows = val + C::kRows + 16 * b;
        const lds_u8 *const tile = at + C::kKey + C::kValue + 32 * group;

        // Operands come out of LDS a step ahead of the products that take them, and products that add to one
        // tile lie apart.
        h8 k[2][4];                            // K of 32 channels: four row tiles
        auto load_k = [&](int d) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const lds_u8 *const from = at + 1024 * (t * kSteps + d) + 8 * lane;
                const u2 lo = lds_get<u2>(from), hi = lds_get<u2>(from + 512);
                k[d & 1][t] = __builtin_bit_cast(h8, u4{lo[0], lo[1], hi[0], hi[1]});
            }
        };
        load_k(0);
        u2 V[4];
        f4 off[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) V[t] = read_column(tile + (16 * t + 4 * b + (m >> 2)) * kColumnBytes + 8 * (m & 3));
#pragma unroll
        for (int t = 0; t < 4; ++t) off[t] = lds_get<f4>(rows + C::kOff + 64 * t);
        const float gamma = lds_get<float>(val + C::kRows + C::kLast);
        const int weigh_up = lds_get<int>(val + C::kRows + C::kLast + 4);
        const f4 heavy = lds_get<f4>(rows + C::kHeavy);

        // ---- K S ----
        f4 ks[4];
        h8 th[6], tl[6];
        auto load_t = [&] {
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                th[i] = lds_get<h8>(val + C::kHigh + 1024 * i + 16 * lane);
                tl[i] = lds_get<h8>(val + C::kLow + 1024 * i + 16 * lane);
            }
        };
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < kSteps; ++d) {
            if (d + 1 < kSteps) {
                load_k(d + 1);
            } else if constexpr (!WARY) {
                load_t();
            }
            const Split x = split(S[2 * d], S[2 * d + 1], 1.0f);
            if (!WARY || !again) lds_put(hand + 1024 * d + 16 * lane, x.hi);
#pragma unroll
            for (int t = 0; t < 4; ++t) ks[t] = mfma16x16x32(k[d & 1][t], x.hi, ks[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t) ks[t] = mfma16x16x32(k[d & 1][t], x.lo, ks[t]);
        }
        if (!WARY || !again) lds_barrier();    // (1) the state is handed over
        float top_s = 0.f;                     // for the next S
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) top_s = __builtin_elementwise_maximum(top_s, __builtin_fabsf(S[t][j]));
        top_s = gamma * top_of_column(top_s);

        // ---- R = V - e^G K S, its rows as operands ----
        const float of_s = times2(1.0f, -power);
        f4 R[4];
        float top_r = 0.f, least = __builtin_inff();
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v = j & 1 ? hi_f32<BF>(V[t][j >> 1]) : lo_f32<BF>(V[t][j >> 1]);
                R[t][j] = __builtin_fmaf(-(off[t][j] * of_s), ks[t][j], v);
                top_r = __builtin_elementwise_maximum(top_r, __builtin_fabsf(R[t][j]));
                least = fminf(least, __builtin_fabsf(R[t][j]));
            }
        top_r = top_of_column(top_r);
        uint64_t lost = 0;                     // rows that come after one that is not finite
        // Sizes far apart, such as factors of them leave fp32, or what is not finite.  (By the last rows alone whether the
        // next state's are large enough: that is where most heads have their heaviest.)
        float of_last = __builtin_fabsf(R[3][0]) * heavy[0];
#pragma unroll
        for (int j = 1; j < 4; ++j) of_last = fmaxf(of_last, __builtin_fabsf(R[3][j]) * heavy[j]);
        const uint64_t enough = __builtin_amdgcn_ballot_w64(of_last >= kSmall * top_r);
        const uint64_t odd = __builtin_amdgcn_ballot_w64(least < kLost * top_r || !(top_r < 0x1p100f) ||
                                                         (top_r < 0x1p-100f && top_r > 0.f) || power < kTop - 100);
        const bool look = odd || ((enough | enough >> 16 | enough >> 32 | enough >> 48) & 0xFFFF) != 0xFFFF;
        if (WARY && look) {
            // (opaque: what is made of it is not kept in registers through the other loop)
            int lane = threadIdx.x & 63;
            asm volatile("" : "+v"(lane));
            const int b = lane >> 4;
            const lds_u8 *const rows = val + C::kRows + 16 * b;
            if (__builtin_amdgcn_ballot_w64(!(top_r < __builtin_inff()))) {
                uint64_t found = 0;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        found |= __builtin_fabsf(R[t][j]) < __builtin_inff() ? 0ull : 1ull << (16 * t + 4 * b + j);
                found |= __shfl_xor(found, 16);
                found |= __shfl_xor(found, 32);
                lost = found ? ~0ull << __builtin_ctzll(found) : 0ull;
                top_r = 0.f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        R[t][j] = lost >> (16 * t + 4 * b + j) & 1 ? 0.f : R[t][j];
                        top_r = fmaxf(top_r, __builtin_fabsf(R[t][j]));
                    }
                top_r = fmaxf(top_r, __shfl_xor(top_r, 16));
                top_r = fmaxf(top_r, __shfl_xor(top_r, 32));
            }
            const int n = min(kChunk, s.n - first - kChunk * ci);
            bool alone = lose(R, times2(1.0f, kTop - max(exponent(top_r), -100)), rows, gamma,
                              times2(top_s, kTop - max(exponent(top_r), -100) + weigh_up - power),
                              lost ? min(n, (int)__builtin_ctzll(lost)) : n, lane, b);
            alone |= top_r >= 0x1p100f || top_r < 0x1p-100f || power < kTop - 100;
            alone = (alone && top_r > 0.f) || lds_get<int>(val + C::kRows + C::kLast + 8) != 0;
            if (__builtin_amdgcn_ballot_w64(alone)) {
                lds_put(factors + 64, kWalked);
                lds_put(lost_at, ~(uint64_t)0);
                lds_barrier();                 // (2) as below
                walk(ci);
                return true;
            }
        }
        if constexpr (WARY) {
            asm volatile("" ::: "memory");     // (not before: registers are short there)
            load_t();
        }
        const int up_r = kTop - max(exponent(top_r), -100);
        const float by_r = times2(1.0f, up_r);

        // ---- U = T R (times 2^(up_r + a power for each row)) ----
        f4 U[4], weigh[4];
        // K^T: four tokens of a channel at a time out of K's operands
        h8 kt[kRowTiles][2];
        auto load_kt = [&](int t) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                u2 part[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int from = 1024 * ((2 * d + e) * kSteps + t / 2) + 512 * (t & 1);
                    part[e] = read_column(at + from + 8 * (16 * (m & 3) + 4 * b + (m >> 2)));
                }
                kt[t][d] = __builtin_bit_cast(h8, u4{part[0][0], part[0][1], part[1][0], part[1][1]});
            }
        };
#pragma unroll
        for (int t = 0; t < 4; ++t) weigh[t] = lds_get<f4>(rows + C::kWeigh + 64 * t);
        {
            const Split r0 = split(R[0], R[1], by_r), r1 = split(R[2], R[3], by_r);
#pragma unroll
            for (int t = 0; t < kRowTiles; ++t) load_kt(t);
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int t = 2 * d; t < 4; ++t) {
                        const Split &r = d ? r1 : r0;
                        U[t] = mfma16x16x32(part < 2 ? th[tile_of(t, d)] : tl[tile_of(t, d)], part == 1 ? r.lo : r.hi, U[t]);
                    }
        }
        if (!WARY && look) return false;       // (here, where the products above hide what this waits for)
#pragma unroll
        for (int t = 0; t < 4; ++t) lds_put(hand + kU + 1024 * t + 16 * lane, U[t]);
        lds_put(factors, of_s);
        lds_put(factors + 64, up_r);
        lds_put(lost_at, lost);
        lds_barrier();                         // (2) and U, and the next chunk is there

        // ---- S <- e^G_last S + (e^(G_last - G) K)^T U ----
        {
            float top_u = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    U[t][j] *= weigh[t][j];
                    top_u = fmaxf(top_u, __builtin_fabsf(U[t][j]));
                }
            top_u = top_of_column(top_u);
            // A power of two for the next S, which has at most 2^14 from this one and 2^15 from the weighed U: 64
            // products of K^T (below 1) and rows below 2^9.  It goes by the largest of them as they are: R's largest
            // may be a row that counts for nothing at the chunk's end.
            const int base = up_r + weigh_up;
            const int next = min(min(kTop + power - (top_s > 0.f ? exponent(top_s) : -200),
                                     kTopU + base - (top_u > 0.f ? max(exponent(top_u), -100) : -200)), power + 100);
            const float by_u = times2(1.0f, next - base);
            const Split u0 = split(U[0], U[1], by_u), u1 = split(U[2], U[3], by_u);
            const float by = times2(gamma, next - power);
            power = next;
#pragma unroll
            for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[t][j] *= by;
#pragma unroll
            for (int part = 0; part < 4; ++part)
#pragma unroll
                for (int t = 0; t < kRowTiles; ++t)
                    S[t] = mfma16x16x32(kt[t][part & 1], part == 0 ? u0.hi : part == 1 ? u1.hi : part == 2 ? u0.lo : u1.lo, S[t]);
            if (WARY && __builtin_amdgcn_ballot_w64(lost != 0)) {
#pragma unroll
                for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t][j] = lost ? __builtin_nanf("") : S[t][j];
            }
        }
        return true;
    };
    lds_barrier();                             // (0) the first chunk is there
    // Whole chunks of ordinary numbers, in a loop of their own, so that its registers stay where they are, and
    // the others.
    const int whole = min(count, (s.n - first) / kChunk);
    for (int ci = 0; ci < count; ++ci) {
        bool again = false;
        while (ci < whole) {
            again = !one_chunk(std::false_type{}, ci, false);
            if (again) break;
            ++ci;
        }
        if (ci < count) one_chunk(std::true_type{}, ci, again);
    }
    {
        if (s.state < 0 && s.n - first <= kChunk * seg.chunks) return;     // (kept for the next segment only)
        float *const to = pool + (int64_t)(4 * b) * a.value_dim + col;
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) to[(int64_t)(16 * t + j) * a.value_dim] = times2(S[t][j], -power);
    }
}

size_t key_bytes(const DeltaArgs &a) { return a.key_dim == 64 ? Chunk<true, 64>::kKey : Chunk<true, 128>::kKey; }
size_t value_bytes(const DeltaArgs &a) { return a.bf16 ? Chunk<true, 128>::kValue : Chunk<false, 128>::kValue; }
size_t chunk_bytes(const DeltaArgs &a) { return a.k_heads * key_bytes(a) + a.v_heads * value_bytes(a); }
int chunks_of(const DeltaArgs &a) { return (a.s.max_q + kChunk - 1) / kChunk; }

// Chunks that the workspace holds at a time.
size_t slots_of(const DeltaArgs &a) {
    constexpr size_t kMost = (size_t)256 << 20;
    return std::max<size_t>(1, kMost / chunk_bytes(a));
}

// How a call is cut: sequences and chunks of each that the workspace holds at a time.
struct Cut {
    int batch, chunks;
};
Cut cut_of(const DeltaArgs &a) {
    const size_t slots = slots_of(a);
    Cut c;
    c.chunks = (int)std::min<size_t>(chunks_of(a), slots);
    c.batch = (int)std::min<size_t>(a.s.batch, std::max<size_t>(1, slots / c.chunks));
    return c;
}

template <bool BF, int DK>
hipError_t launch_row(const DeltaArgs &a, hipStream_t stream) {
    const Cut c = cut_of(a);
    Segment seg;
    seg.keys = static_cast<uint8_t *>(a.workspace);
    seg.values = seg.keys + (size_t)c.chunks * c.batch * a.k_heads * Chunk<BF, DK>::kKey;
    seg.carry = reinterpret_cast<float *>(seg.values + (size_t)c.chunks * c.batch * a.v_heads * Chunk<BF, DK>::kValue);
    for (int b0 = 0; b0 < a.s.batch; b0 += c.batch) {
        for (int c0 = 0; c0 < chunks_of(a); c0 += c.chunks) {
            seg.first_seq = b0;
            seg.batch = std::min(c.batch, a.s.batch - b0);
            seg.first_chunk = c0;
            seg.chunks = std::min(c.chunks, chunks_of(a) - c0);
            // Value heads that share a key head in one workgroup, as long as that leaves two for every CU (one sequence of
            // 8191 tokens, 16 + 48 heads, the whole call: 307 us, each alone 323; 8 of 500: 127 and 139; but one of
            // 1000, 768 workgroups: 58.5 together, 53.2 alone).
            int heads = 1;
            for (int i = 2; i <= kMostHeads; ++i)
                if (a.v_heads / a.k_heads % i == 0 && (int64_t)seg.chunks * a.v_heads / i * seg.batch >= 512) heads = i;
            chunk_prep_kernel<BF, DK, false><<<dim3(seg.chunks, a.v_heads / heads, seg.batch), 256, 0, stream>>>(a, seg, heads);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            // 32 columns a workgroup while each finds a CU of its own, else 64 (the whole call: one sequence of 8191 tokens, 48
            // heads, 192 workgroups 307 and 386 us; two of 4000, 32 heads, 256: 144 and 159; two of 2000, 48 heads, 384:
            // 159 and 124; five of 2500, 32 heads: 273 and 228).
            if ((int64_t)a.value_dim / 32 * a.v_heads * seg.batch <= 256)
                chunk_scan_kernel<BF, DK, 2><<<dim3(a.value_dim / 32, a.v_heads, seg.batch), 256, 0, stream>>>(a, seg);
            else
                chunk_scan_kernel<BF, DK, 4><<<dim3(a.value_dim / 64, a.v_heads, seg.batch), 512, 0, stream>>>(a, seg);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

template <bool BF, int DK>
hipError_t launch_tree(const DeltaArgs &a, hipStream_t stream) {
    Segment seg{};
    seg.batch = a.s.batch;
    seg.chunks = 1;
    chunk_prep_kernel<BF, DK, true><<<dim3(1, a.v_heads, a.s.batch), 256, 0, stream>>>(a, seg, 1);
    return hipGetLastError();
}

}  // namespace

size_t delta_chunk_workspace_bytes(const DeltaArgs &a) {
    if (a.s.tree) return 0;
    const Cut c = cut_of(a);
    // (not by how this call is cut: a smaller one may fill more of what there is at a time)
    size_t bytes = chunk_bytes(a) * std::min<size_t>(slots_of(a), (size_t)chunks_of(a) * a.s.batch);
    if (c.chunks < chunks_of(a)) bytes += (size_t)c.batch * a.v_heads * a.key_dim * a.value_dim * 4;
    return bytes;
}

hipError_t launch_delta_chunk(const DeltaArgs &a, hipStream_t stream) {
    auto go = [&](auto bf, auto dk) {
        return a.s.tree ? launch_tree<bf(), dk()>(a, stream) : launch_row<bf(), dk()>(a, stream);
    };
    auto sized = [&](auto bf) {
        return a.key_dim == 64 ? go(bf, std::integral_constant<int, 64>{}) : go(bf, std::integral_constant<int, 128>{});
    };
    return a.bf16 ? sized(std::true_type{}) : sized(std::false_type{});
}

}  // namespace w4a16
