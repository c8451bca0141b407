// Keys and values into the 4-bit cache and back, and the norm and rotation of
// queries and keys on the way.
//
//   y = x / sqrt(mean(x^2) + eps) * w        over the D channels of a head
//   (a, b) -> (a cos - b sin, b cos + a sin)  for the pairs of the first rot
//                                             channels: (i, i + rot/2), or
//                                             (2i, 2i + 1) when interleaved
//   m = round(min), s = round((max - min) * (1/15)), c = rint((y - m) * (1/s))
// per group of g channels, s and m in the activation type, everything else in
// fp32; the stored value is m + s c.  A group with a value that is not finite,
// or whose s or m is not, is stored as NaN (s = m = NaN).
//
// All of it is bound by memory traffic (about 10 flops a channel).  A head is
// spread over D/8 lanes with eight neighbouring channels each: one 16-byte
// load, the sum of squares and the group's extremes by shuffles within those
// lanes, and a lane's eight codes are exactly one key word of the cache.
// Measured (fp16 or bfloat16): norm and rotation of the 170 MB of a prompt in and
// out 40 us (4.3 TB/s; a copy reaches 5.2), of one token 2.9; into the cache one
// token of each of 64 sequences 6.5 us (a chain of four loads), three chunks of
// prompts 25.2 and their rows back 10.9 (95 MB together, 2.6 TB/s).

#include "kv4_device.hpp"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

// Eight 16-bit values as fp32.
template <bool BF>
__device__ __forceinline__ void widen(u4 v, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = lo_f32<BF>(v[j]);
        x[2 * j + 1] = hi_f32<BF>(v[j]);
    }
}

template <bool BF>
__device__ __forceinline__ u4 narrow(const float (&x)[8]) {
    return u4{pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3]), pack2<BF>(x[4], x[5]), pack2<BF>(x[6], x[7])};
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
    }
}

// 1 / sqrt(v) rounded to nearest: one Newton step in fp64 on the hardware's approximation, which
// is off by an ulp for a ninth of all arguments.  A head's channels all share this factor, and a
// stored code should not turn on its last bit.
__device__ __forceinline__ float inverse_root(float v) {
    const double r = (double)__builtin_amdgcn_rsqf(v);
    return (float)(r * (1.5 - 0.5 * (double)v * r * r));
}

// Norm and rotation of channels 8 i .. 8 i + 7 of a head whose D/8 lanes call
// this together.  pos: the token's position; one outside the tables gives NaN.
// No contraction: the products and sums round as the formulas above say.
template <int D>
__device__ __forceinline__ void norm_rope(float (&x)[8], int i, const float *weight, const RopeArgs &r,
                                          int pos) {
#pragma clang fp contract(off)
    if (weight) {
        // fours, then a balanced tree: the order of the error of a sum of D terms is log2 D
        float sum = (((x[0] * x[0] + x[1] * x[1]) + x[2] * x[2]) + x[3] * x[3]) +
                    (((x[4] * x[4] + x[5] * x[5]) + x[6] * x[6]) + x[7] * x[7]);
#pragma unroll
        for (int d = 1; d < D / 8; d *= 2) sum += __shfl_xor(sum, d);
        float rstd;
        if (__builtin_expect(sum < 0x1p126f && sum + r.eps > 0x1p-90f, 1)) {
            rstd = inverse_root(sum * (1.0f / D) + r.eps);
        } else {
            // squares that leave fp32 (bfloat16 beyond 1e19 or below 1e-14, or all zeros): in 64 bits
            double squares = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) squares += (double)x[j] * x[j];
#pragma unroll
            for (int d = 1; d < D / 8; d *= 2) squares += __shfl_xor(squares, d);
            rstd = (float)(1.0 / sqrt(squares * (1.0 / D) + (double)r.eps));
        }
        float w[8];
        load8(weight + 8 * i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * rstd * w[j];
    }
    if (!r.cos) return;
    const bool inside = (unsigned)pos < (unsigned)r.max_pos;
    const int half = r.rot / 2;
    const int64_t row = (int64_t)(inside ? pos : 0) * half;
    if (r.interleaved) {
        if (8 * i < r.rot) {
            const f4 c = *reinterpret_cast<const f4 *>(r.cos + row + 4 * i);
            const f4 s = *reinterpret_cast<const f4 *>(r.sin + row + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * c[j] - b * s[j];
                x[2 * j + 1] = b * c[j] + a * s[j];
            }
        }
    } else {
        // the partner channels are rot/16 lanes away; every lane takes part in the shuffles
        const int lanes = half / 8;
        const bool rotated = 8 * i < r.rot, first = i < lanes;
        const int from = (int)(threadIdx.x & 63) + (rotated ? (first ? lanes : -lanes) : 0);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __shfl(x[j], from);
        if (rotated) {
            float c[8], s[8];
            load8(r.cos + row + 8 * (first ? i : i - lanes), c);
            load8(r.sin + row + 8 * (first ? i : i - lanes), s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = o[j] * s[j];
                x[j] = first ? x[j] * c[j] - t : x[j] * c[j] + t;
            }
        }
    }
    if (!inside) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
    }
}

// Codes of a lane's eight channels (channel 8 i + j in codes[j]) and the
// group's parameter word; the G/8 lanes of a group call this together.
template <bool BF, int G>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t (&codes)[8]) {
#pragma clang fp contract(off)
    float lo = x[0], hi = x[0];
    bool bad = !(fabsf(x[0]) < __builtin_inff());
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
        bad |= !(fabsf(x[j]) < __builtin_inff());
    }
#pragma unroll
    for (int d = 1; d < G / 8; d *= 2) {
        lo = fminf(lo, __shfl_xor(lo, d));
        hi = fmaxf(hi, __shfl_xor(hi, d));
        bad |= __shfl_xor((int)bad, d) != 0;
    }
    uint32_t par = pack2<BF>((hi - lo) * (1.0f / 15.0f), lo);
    float s = par_step<BF>(par), m = par_offset<BF>(par);
    // a value that is not finite, or a step or offset that the type does not hold: NaN
    if (bad || !(s < __builtin_inff()) || !(fabsf(m) < __builtin_inff())) {
        s = m = __builtin_nanf("");
        par = pack2<BF>(s, m);
    }
    // a step below the normal range has no reciprocal: the group is its offset
    const float inv = s >= 1.17549435e-38f ? 1.0f / s : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float c = fminf(fmaxf(rintf((x[j] - m) * inv), 0.0f), 15.0f);
        codes[j] = (uint32_t)(int)c;
    }
    return s >= 1.17549435e-38f || s != s ? par : par & 0xFFFF0000u;
}

template <bool BF, int D>
__device__ __forceinline__ void head_row(const HeadsArgs &a, const RopeArgs &r, int64_t token, int h,
                                         int i) {
    constexpr int kStep = D;
    const uint16_t *src = static_cast<const uint16_t *>(a.x) + token * a.x_stride + h * kStep + 8 * i;
    float x[8];
    widen<BF>(*reinterpret_cast<const u4 *>(src), x);
    norm_rope<D>(x, i, a.weight, r, r.cos ? r.positions[token] : 0);
    uint16_t *dst = static_cast<uint16_t *>(a.y) + token * a.y_stride + h * kStep + 8 * i;
    *reinterpret_cast<u4 *>(dst) = narrow<BF>(x);
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(HeadsArgs q, HeadsArgs k, RopeArgs r,
                                                             int64_t rows) {
    constexpr int kLanes = D / 8;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (row >= rows) return;
    const int heads = q.heads + k.heads;
    const int64_t token = row / heads;
    const int h = (int)(row - token * heads);
    const int i = threadIdx.x % kLanes;
    if (h < q.heads)
        head_row<BF, D>(q, r, token, h, i);
    else
        head_row<BF, D>(k, r, token, h - q.heads, i);
}

// One workgroup: the new slots of one tile of one head (blocks below
// tile_blocks), or rows of query heads.  A workgroup owns its tile, so a
// value word that several new slots share is put together in LDS and written
// once; nibbles of older slots in it are read and kept.
template <bool BF, int D, int NG>
__global__ void __launch_bounds__(kThreads) append_kernel(Kv4AppendArgs a, int tiles, int tile_blocks) {
    constexpr int kLanes = D / 8;
    using T = Tile<D, NG>;
    if ((int)blockIdx.x >= tile_blocks) {
        const int64_t row = (int64_t)((int)blockIdx.x - tile_blocks) * (kThreads / kLanes) +
                            threadIdx.x / kLanes;
        const int64_t token = row / a.q.heads;
        if (token < a.T)
            head_row<BF, D>(a.q, a.r, token, (int)(row - token * a.q.heads), threadIdx.x % kLanes);
        return;
    }
    __shared__ __align__(16) uint8_t codes[32 * D];
    const int h = blockIdx.x % a.c.kv_heads;
    const int rest = blockIdx.x / a.c.kv_heads;
    const int b = rest / tiles;
    const int64_t first = a.cu[b], end = a.cu[b + 1];
    const int64_t n64 = min(end, a.T) - first;
    if (first < 0 || n64 <= 0) return;
    // slots of the first new token, and after the last one that max_q leaves
    const int64_t start64 = (int64_t)a.kv_len[b] - (end - first);
    const int64_t base64 = 32 * ((start64 >> 5) + rest % tiles);
    const int stop = (int)min(start64 + min(n64, (int64_t)a.max_q), (int64_t)0x7fffffff);
    if (base64 < 0 || base64 >= stop) return;
    const int start = (int)start64, base = (int)base64, tile = base >> 5;
    uint8_t *p = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b, h, tile);
    if (!p) return;
    const int lo = max(start - base, 0), hi = min(stop - base, 32), count = hi - lo;
    uint32_t *words = reinterpret_cast<uint32_t *>(p);
    uint32_t *params = reinterpret_cast<uint32_t *>(p + 2 * T::kCodes);
    for (int idx = threadIdx.x; idx < 2 * count * kLanes; idx += kThreads) {
        const int i = idx % kLanes;
        const bool value = idx >= count * kLanes;
        const int r32 = lo + idx / kLanes - (value ? count : 0);
        const int64_t token = first + (base + r32 - start);
        const HeadsArgs &src = value ? a.v : a.k;
        float x[8];
        widen<BF>(*reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(src.x) +
                                                token * src.x_stride + h * D + 8 * i), x);
        if (!value) norm_rope<D>(x, i, a.k.weight, a.r, a.r.cos ? a.r.positions[token] : 0);
        uint32_t c[8];
        const uint32_t par = quantise<BF, T::kGroup>(x, c);
        if (i % (T::kGroup / 8) == 0)
            params[(value ? 32 * NG : 0) + 32 * (i / (T::kGroup / 8)) + r32] = par;
        if (value) {
            *reinterpret_cast<u2 *>(codes + r32 * D + 8 * i) =
                u2{c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
        } else {
            words[key_word<D>(r32, i)] = c[0] | c[2] << 4 | c[4] << 8 | c[6] << 12 | c[1] << 16 |
                                         c[3] << 20 | c[5] << 24 | c[7] << 28;
        }
    }
    __syncthreads();
    words += T::kCodes / 4;
    for (int at = threadIdx.x; at < 4 * D; at += kThreads) {
        const int lane = (at >> 2) & 63;
        const int d = 16 * (4 * (at >> 8) + (at & 3)) + (lane & 15);
        uint32_t mask = 0, w = 0;
#pragma unroll
        for (int nib = 0; nib < 8; ++nib) {
            const int r32 = 4 * (lane >> 4) + (nib & 3) + 16 * (nib >> 2);
            if (r32 >= lo && r32 < hi) {
                mask |= 0xFu << (4 * nib);
                w |= (uint32_t)codes[r32 * D + d] << (4 * nib);
            }
        }
        if (mask == 0) continue;
        if (mask != 0xFFFFFFFFu) w |= words[at] & ~mask;
        words[at] = w;
    }
}

// Rows of one head: the last cu[b + 1] - cu[b] slots of each sequence b, as values m + s c (exact
// in fp32 up to one rounding) rounded to the activation type.  A workgroup takes 32 rows.  Where
// they are one sequence's, the two tiles that they lie in are copied to LDS whole (16-byte
// loads, each word once for the eight slots in it); else each row reads its own words.
constexpr int kSearch = 1024;      // sequences whose ends fit LDS
template <bool BF, int D, int NG>
__global__ void __launch_bounds__(kThreads) read_kernel(Kv4ReadArgs a) {
    constexpr int kLanes = D / 8;
    using T = Tile<D, NG>;
    __shared__ __align__(16) uint8_t tiles[2 * T::kBytes];
    __shared__ int ends[kSearch];
    const int h = blockIdx.y, batch = a.c.batch;
    const int64_t row0 = (int64_t)blockIdx.x * 32;
    const bool in_lds = batch <= kSearch;
    if (in_lds) {
        for (int b = threadIdx.x; b < batch; b += kThreads) ends[b] = a.cu[b + 1];
        __syncthreads();
    }
    // the sequence that a row belongs to: the first that ends after it
    auto sequence_of = [&](int64_t row) {
        int lo = 0, hi = batch;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if ((in_lds ? ends[mid] : a.cu[mid + 1]) <= row)
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo;
    };
    const int64_t last = min(row0 + 31, a.rows - 1);
    const int b0 = __builtin_amdgcn_readfirstlane(sequence_of(row0));
    const int64_t end0 = b0 < batch ? a.cu[b0 + 1] : 0;
    const int slot0 = b0 < batch ? a.kv_len[b0] - (int)(end0 - row0) : 0;
    const bool one = b0 < batch && last < end0 && slot0 >= 0;      // all rows are b0's, from slot0 on
    const uint8_t *from0 = nullptr, *from1 = nullptr;
    if (one) {
        from0 = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b0, h, slot0 >> 5);
        from1 = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b0, h, (slot0 >> 5) + 1);
        for (int i = threadIdx.x; i < T::kBytes / 16; i += kThreads) {
            if (from0) reinterpret_cast<u4 *>(tiles)[i] = reinterpret_cast<const u4 *>(from0)[i];
            if (from1 && slot0 % 32) reinterpret_cast<u4 *>(tiles + T::kBytes)[i] = reinterpret_cast<const u4 *>(from1)[i];
        }
        __syncthreads();
    }
    for (int idx = threadIdx.x; idx < 32 * kLanes; idx += kThreads) {
        const int64_t row = row0 + idx / kLanes;
        const int i = idx % kLanes;
        if (row >= a.rows) return;
        const uint8_t *p;
        int slot;
        if (one) {
            slot = slot0 + idx / kLanes;
            const bool second = (slot >> 5) != (slot0 >> 5);
            p = (second ? from1 : from0) ? tiles + (second ? T::kBytes : 0) : nullptr;
        } else {
            const int b = sequence_of(row);
            if (b >= batch) return;
            slot = a.kv_len[b] - (int)(a.cu[b + 1] - row);
            p = slot < 0 ? nullptr : tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b, h, slot >> 5);
        }
        const int r32 = slot & 31, g = 8 * i / T::kGroup;
        float k[8], v[8];
        if (p) {
            const uint32_t *words = reinterpret_cast<const uint32_t *>(p);
            const uint32_t *params = reinterpret_cast<const uint32_t *>(p + 2 * T::kCodes);
            const uint32_t kp = params[32 * g + r32], vp = params[32 * (NG + g) + r32];
            const uint32_t kw = words[key_word<D>(r32, i)];
            words += T::kCodes / 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t ck = (kw >> (4 * (j >> 1) + 16 * (j & 1))) & 15u;
                const uint32_t cv = (words[value_word(r32, 8 * i + j)] >> value_shift(r32)) & 15u;
                k[j] = __builtin_fmaf(par_step<BF>(kp), (float)ck, par_offset<BF>(kp));
                v[j] = __builtin_fmaf(par_step<BF>(vp), (float)cv, par_offset<BF>(vp));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = v[j] = __builtin_nanf("");
        }
        const int64_t at = (row * a.c.kv_heads + h) * D + 8 * i;
        *reinterpret_cast<u4 *>(static_cast<uint16_t *>(a.k) + at) = narrow<BF>(k);
        *reinterpret_cast<u4 *>(static_cast<uint16_t *>(a.v) + at) = narrow<BF>(v);
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

hipError_t launch_qk_norm_rope(const HeadsArgs &q, const HeadsArgs &k, const RopeArgs &r, int64_t T,
                               int head_dim, bool bf16, hipStream_t stream) {
    const int64_t rows = T * (q.heads + k.heads);
    const int per = kThreads / (head_dim / 8);
    const dim3 grid((unsigned)((rows + per - 1) / per));
    auto go = [&](auto bf, auto d) {
        norm_rope_kernel<bf(), d()><<<grid, kThreads, 0, stream>>>(q, k, r, rows);
        return hipGetLastError();
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    using I256 = std::integral_constant<int, 256>;
    auto typed = [&](auto d) { return bf16 ? go(std::true_type{}, d) : go(std::false_type{}, d); };
    return head_dim == 64 ? typed(I64{}) : head_dim == 128 ? typed(I128{}) : typed(I256{});
}

hipError_t launch_kv4_append(const Kv4AppendArgs &a, hipStream_t stream) {
    const int tiles = (a.max_q + 62) / 32;       // tiles that max_q new slots can touch
    const int64_t tile_blocks = (int64_t)a.c.batch * tiles * a.c.kv_heads;
    const int per = kThreads / (a.c.head_dim / 8);
    const int64_t blocks = tile_blocks + (a.T * a.q.heads + per - 1) / per;
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        append_kernel<bf(), d(), ng()><<<dim3((unsigned)blocks), kThreads, 0, stream>>>(
            a, tiles, (int)tile_blocks);
        return hipGetLastError();
    });
}

hipError_t launch_kv4_read(const Kv4ReadArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.rows + 31) / 32), (unsigned)a.c.kv_heads);
    return by_shape(a.c, [&](auto bf, auto d, auto ng) {
        read_kernel<bf(), d(), ng()><<<grid, kThreads, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace w4a16
