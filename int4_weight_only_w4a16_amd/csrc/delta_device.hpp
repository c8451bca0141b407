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

}  // namespace w4a16
