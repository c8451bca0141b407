// What the kernels of the gated delta rule and the short convolution share.
#pragma once

#include "delta_launch.h"
#include "w4a16_device.hpp"

namespace w4a16 {

// One sequence of a call.
struct Seq {
    int64_t first;       // its first row
    int n;               // rows of this call
    int64_t state;       // its state, or -1: none
    bool fresh;          // the state is taken as zeros
};

__device__ __forceinline__ bool seq_of(const Sequences &s, int b, Seq *q) {
    const int64_t first = s.cu[b], end = min((int64_t)s.cu[b + 1], s.T);
    if (first < 0 || end <= first) return false;
    q->first = first;
    q->n = (int)min(end - first, (int64_t)s.max_q);
    const int i = s.index[b];
    q->state = (unsigned)i < (unsigned)s.num_states ? i : -1;
    q->fresh = q->state < 0 || (s.seen && s.seen[b] <= 0);
    return true;
}

// The gates of one token and head: g, the logarithm of what the state keeps, and beta.
struct Gates {
    float g, beta;
};

// From the projections x = a + dt_bias and b: g = -rate softplus(x), beta = sigmoid(b).
__device__ __forceinline__ Gates gates_from(float a, float b, float rate, float bias) {
    const float x = a + bias;
    // log1p keeps softplus precise where e^x is small, as it is for heads that forget slowly
    const float soft = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    return {x != x ? x : -rate * soft, 1.0f / (1.0f + expf(-b))};
}

template <bool BF>
__device__ __forceinline__ Gates gates_of(const DeltaArgs &a, int64_t row, int h, float rate, float bias) {
    if (!a.a_log)
        return {static_cast<const float *>(a.a)[row * a.a_stride + h], static_cast<const float *>(a.b)[row * a.b_stride + h]};
    return gates_from(lo_f32<BF>(static_cast<const uint16_t *>(a.a)[row * a.a_stride + h]),
                      lo_f32<BF>(static_cast<const uint16_t *>(a.b)[row * a.b_stride + h]), rate, bias);
}

// Sum over the lanes that are equal mod EQUAL, 4 or 16, without LDS.
template <int EQUAL>
__device__ __forceinline__ float over_lanes(float v) {
    static_assert(EQUAL == 4 || EQUAL == 16, "rows of 16 lanes");
#define W4A16_ADD_ROR(N) \
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + N, 0xF, 0xF, true))
    if constexpr (EQUAL == 4) {
        W4A16_ADD_ROR(8);
        W4A16_ADD_ROR(4);
    }
#undef W4A16_ADD_ROR
    const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
    const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}

// x / sqrt(sum x^2 + eps) over the lanes that are equal mod EQUAL and hold one vector; in 64 bits where squares
// leave fp32.
template <int EQUAL, int N>
__device__ __forceinline__ void to_unit(float (&x)[N], float eps) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum = __builtin_fmaf(x[i], x[i], sum);
    sum = over_lanes<EQUAL>(sum) + eps;
    if (sum > 1e-30f && sum < 1e38f) {
        const float f = __builtin_amdgcn_rsqf(sum);        // (within 2^-23)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= f;
        return;
    }
    double wide = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) wide += (double)x[i] * x[i];
#pragma unroll
    for (int d = EQUAL; d < 64; d *= 2) wide += __shfl_xor(wide, d);
    const double f = 1.0 / sqrt(wide + eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)(x[i] * f);
}

}  // namespace w4a16
