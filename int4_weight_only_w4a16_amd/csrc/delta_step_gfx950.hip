// The gated delta rule token by token.
//
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// Both sums over the state come from one pass over the old one:
//   u = beta (v - e^g S^T k),  o = scale (e^g S^T q + (k . q) u),  S <- e^g S + k u^T
// A wave keeps sixteen columns of one head's state in registers: lane 4 r + c has rows
// Dk / 16 r .. of columns 4 c .. 4 c + 3, so that a token costs no barrier and its key and query
// one load in each lane.  Columns do not depend on each other.
// Bound by memory for one token (the state in and out, 2 x 4 Dk Dv bytes a head).

#include <type_traits>

#include "delta_device.hpp"

namespace w4a16 {
namespace {

constexpr int kColumns = 16;

__device__ __forceinline__ float over_rows(float v) {      // sum over the lanes of one column
#pragma unroll
    for (int d = 4; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// x / sqrt(sum x^2 + eps) over the lanes of a column; in 64 bits where squares leave fp32.
template <int N>
__device__ __forceinline__ void to_unit(float (&x)[N], float eps) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum = __builtin_fmaf(x[i], x[i], sum);
    sum = over_rows(sum) + eps;
    if (sum > 1e-30f && sum < 1e38f) {
        const float f = 1.0f / sqrtf(sum);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= f;
        return;
    }
    double wide = 0;
    for (int i = 0; i < N; ++i) wide += (double)x[i] * x[i];
#pragma unroll
    for (int d = 4; d < 64; d *= 2) wide += __shfl_xor(wide, d);
    const double f = 1.0 / sqrt(wide + eps);
    for (int i = 0; i < N; ++i) x[i] = (float)(x[i] * f);
}

template <bool BF, int DK>
__global__ void __launch_bounds__(64) step_kernel(DeltaArgs a) {
    constexpr int kRows = DK / 16;
    const int lane = threadIdx.x, r = lane >> 2, col = blockIdx.x * kColumns + 4 * (lane & 3);
    const int h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
    Seq s;
    if (!seq_of(a.s, blockIdx.z, &s)) return;

    float *const state = a.state + ((max(s.state, (int64_t)0) * a.v_heads + h) * DK + kRows * r) * a.value_dim + col;
    f4 S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        S[i] = s.fresh ? f4{0.f, 0.f, 0.f, 0.f} : *reinterpret_cast<const f4 *>(state + (int64_t)i * a.value_dim);
    const float rate = a.a_log ? expf(a.a_log[h]) : 0.f, bias = a.a_log ? a.dt_bias[h] : 0.f;
    const uint16_t *const q0 = static_cast<const uint16_t *>(a.q) + hk * DK + kRows * r;
    const uint16_t *const k0 = static_cast<const uint16_t *>(a.k) + hk * DK + kRows * r;
    const uint16_t *const v0 = static_cast<const uint16_t *>(a.v) + h * a.value_dim + col;

    auto token = [&](int t) {
        const int64_t row = s.first + t;
        float q[kRows], k[kRows], v[4];
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
            const u2 qq = *reinterpret_cast<const u2 *>(q0 + row * a.q_stride + i);
            const u2 kk = *reinterpret_cast<const u2 *>(k0 + row * a.k_stride + i);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                q[i + 2 * e] = lo_f32<BF>(qq[e]);
                q[i + 2 * e + 1] = hi_f32<BF>(qq[e]);
                k[i + 2 * e] = lo_f32<BF>(kk[e]);
                k[i + 2 * e + 1] = hi_f32<BF>(kk[e]);
            }
        }
        const u2 vv = *reinterpret_cast<const u2 *>(v0 + row * a.v_stride);
        v[0] = lo_f32<BF>(vv[0]);
        v[1] = hi_f32<BF>(vv[0]);
        v[2] = lo_f32<BF>(vv[1]);
        v[3] = hi_f32<BF>(vv[1]);
        const Gates gate = gates_of<BF>(a, row, h, rate, bias);
        const float keep = expf(gate.g);

        if (a.unit) {
            to_unit(k, a.eps);
            to_unit(q, a.eps);
        }
        float qk = 0.f;
        f4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            qk = __builtin_fmaf(q[i], k[i], qk);
            sk += S[i] * k[i];
            sq += S[i] * q[i];
        }
        qk = over_rows(qk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] = over_rows(sk[e]);
            sq[e] = over_rows(sq[e]);
        }
        f4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = gate.beta * (v[e] - keep * sk[e]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i] = keep * S[i] + k[i] * u;
        if (r == 0) {
            const f4 o = a.scale * (keep * sq + qk * u);
            *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + row * a.out_stride + (int64_t)h * a.value_dim + col) =
                pack4<BF>(o[0], o[1], o[2], o[3]);
        }
    };

    for (int t = 0; t < s.n; ++t) token(t);
    if (s.state < 0) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i) *reinterpret_cast<f4 *>(state + (int64_t)i * a.value_dim) = S[i];
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream) {
    const dim3 grid(a.value_dim / kColumns, a.v_heads, a.s.batch);
    auto go = [&](auto bf, auto dk) {
        step_kernel<bf(), dk()><<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    };
    auto typed = [&](auto dk) { return a.bf16 ? go(std::true_type{}, dk) : go(std::false_type{}, dk); };
    return a.key_dim == 64 ? typed(std::integral_constant<int, 64>{}) : typed(std::integral_constant<int, 128>{});
}

}  // namespace w4a16
