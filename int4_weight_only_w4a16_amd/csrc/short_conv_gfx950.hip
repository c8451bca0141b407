// Short causal convolution of every channel over [state, tokens], with SiLU.
//
//   y[t][c] = act(bias[c] + sum_j w[c][j] x[t - (W - 1) + j][c]),  W = 2, 3 or 4
// with the rows before a sequence's first new token from its state (the last W - 1 rows), which
// moves on by the call's tokens.  In a tree of drafts the rows before a token are its ancestors',
// and the state stays.
//
// Bound by memory: 2 bytes in and 2 out a value, and the rows before a block of tokens again
// (from L2).  A lane takes eight channels (16 bytes) of R tokens in a row, all of whose loads are
// under way at once, with one load of the weights (twice the bytes of a token's row); sums are fp32,
// rounded once.  (Three prompts of 1700 to 5001 tokens, 10240 channels: 86 us, 4.8 TB/s; 16 trees of
// 9 to 40 drafts, 8192 channels: 10.0 us with four tokens a lane, 11.4 with two, 12.6 with one; one
// token: 5, of which a launch is the most.)

#include <algorithm>
#include <type_traits>

#include "delta_device.hpp"

namespace w4a16 {
namespace {

constexpr int kLanes = 64;                 // of a wave, 8 channels each

// silu(z) = z / (1 + e^-z); both results of the hardware are off by about 2^-23.
__device__ __forceinline__ float silu_fast(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

template <bool BF>
__device__ __forceinline__ void unpack8(u4 v, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = lo_f32<BF>(v[e]);
        f[2 * e + 1] = hi_f32<BF>(v[e]);
    }
}

template <bool BF, int W, int R, bool TREE>
__global__ void __launch_bounds__(256) conv_kernel(ConvArgs a, int channel_blocks) {
    // (of a sequence only the lane that moves a channel's state on reads it)
    static_assert(TREE || R >= W - 1, "later lanes' rows are all tokens");
    const int cb = blockIdx.x % channel_blocks, tb = blockIdx.x / channel_blocks;
    const int c = 8 * (cb * kLanes + threadIdx.x);
    Seq q;
    if (c >= a.channels || !seq_of(a.s, blockIdx.y, &q)) return;
    if (TREE) q.n = min(q.n, 64);
    const int t0 = (tb * blockDim.y + threadIdx.y) * R;
    if (t0 >= q.n) return;

    const uint16_t *const x = static_cast<const uint16_t *>(a.x) + q.first * a.x_stride + c;
    uint16_t *const state = static_cast<uint16_t *>(a.state) + max(q.state, (int64_t)0) * (W - 1) * a.channels + c;
    const u4 none = {0u, 0u, 0u, 0u};
    // row p of [state, tokens]: p < 0 is the state's
    auto row = [&](int p) {
        if (p >= 0) return *reinterpret_cast<const u4 *>(x + (int64_t)p * a.x_stride);
        return q.fresh ? none : *reinterpret_cast<const u4 *>(state + (int64_t)(W - 1 + p) * a.channels);
    };
    float w[8][W], bias[8];
    {
        const f4 *const from = reinterpret_cast<const f4 *>(a.weight + (int64_t)c * W);
        float flat[8 * W];
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            const f4 v = from[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) flat[4 * i + e] = v[e];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = flat[i * W + j];
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = 0.f;
        if (a.bias) {
            const f4 b0 = *reinterpret_cast<const f4 *>(a.bias + c), b1 = *reinterpret_cast<const f4 *>(a.bias + c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bias[i] = b0[i];
                bias[4 + i] = b1[i];
            }
        }
    }
    auto put = [&](int t, const u4 (&rows)[W]) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float f[8];
            unpack8<BF>(rows[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w[i][j], f[i], y[i]);
        }
        if (a.silu)
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = silu_fast(y[i]);
        u4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack2<BF>(y[2 * e], y[2 * e + 1]);
        *reinterpret_cast<u4 *>(static_cast<uint16_t *>(a.out) + (q.first + t) * a.out_stride + c) = o;
    };

    if constexpr (TREE) {
        uint64_t word[R];
#pragma unroll
        for (int r = 0; r < R; ++r) word[r] = (uint64_t)a.s.tree[q.first + min(t0 + r, q.n - 1)];
        u4 rows[R][W];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int p = min(t0 + r, q.n - 1);
            word[r] &= (1ull << p) - 1;
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                rows[r][j] = row(p);
                // the latest token that this one descends from; then back through the state
                if (word[r]) {
                    p = 63 - __clzll(word[r]);
                    word[r] &= ~(1ull << p);
                } else {
                    p = min(p, 0) - 1;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (t0 + r >= q.n) return;
            put(t0 + r, rows[r]);
        }
        return;
    }
    u4 rows[W - 1 + R];
#pragma unroll
    for (int j = 0; j < W - 1 + R; ++j) {
        const int p = t0 - (W - 1) + j;
        rows[j] = p < q.n ? row(p) : none;
    }
    if (t0 == 0 && q.state >= 0) {
        // the state moves on; of a sequence its old rows are read here and nowhere else
        u4 last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = row(q.n - (W - 1) + j);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<u4 *>(state + (int64_t)j * a.channels) = last[j];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (t0 + r >= q.n) return;
        u4 at[W];
#pragma unroll
        for (int j = 0; j < W; ++j) at[j] = rows[r + j];
        put(t0 + r, at);
    }
}

// Tokens of a lane, and token blocks of a workgroup.  Without a tree four tokens a lane for short calls, for more lanes, else
// eight, for fewer loads of weights and rows (10240 channels, us with four and eight: 4 sequences of 20 tokens 5.0 and
// 5.5, 16 of 40 with 8192 8.9 and 9.4; of 64 tokens one 5.0 and 5.8, but 4 6.8 and 6.4, 16 12.2 and 10.6; 3 of 4000
// 119 and 101).
constexpr int kTreeTokens = 4;
int tokens_of(const ConvArgs &a) { return a.s.tree ? kTreeTokens : a.s.max_q < 64 ? 4 : 8; }
int rows_of(const ConvArgs &a) { return std::min(4, (a.s.max_q + tokens_of(a) - 1) / tokens_of(a)); }
int64_t channel_blocks(const ConvArgs &a) { return (a.channels + 8 * kLanes - 1) / (8 * kLanes); }

}  // namespace

int conv_threads(const ConvArgs &a) { return kLanes * rows_of(a); }
int64_t conv_blocks(const ConvArgs &a) {
    const int64_t per = (int64_t)rows_of(a) * tokens_of(a);
    return channel_blocks(a) * ((a.s.max_q + per - 1) / per);
}

hipError_t launch_short_conv(const ConvArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)conv_blocks(a), (unsigned)a.s.batch), block(kLanes, rows_of(a));
    const int cbs = (int)channel_blocks(a);
    auto go = [&](auto bf, auto w) {
        if (a.s.tree)
            conv_kernel<bf(), w(), kTreeTokens, true><<<grid, block, 0, stream>>>(a, cbs);
        else if (tokens_of(a) == 4)
            conv_kernel<bf(), w(), 4, false><<<grid, block, 0, stream>>>(a, cbs);
        else
            conv_kernel<bf(), w(), 8, false><<<grid, block, 0, stream>>>(a, cbs);
        return hipGetLastError();
    };
    auto typed = [&](auto w) { return a.bf16 ? go(std::true_type{}, w) : go(std::false_type{}, w); };
    switch (a.width) {
        case 2: return typed(std::integral_constant<int, 2>{});
        case 3: return typed(std::integral_constant<int, 3>{});
        case 4: return typed(std::integral_constant<int, 4>{});
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
