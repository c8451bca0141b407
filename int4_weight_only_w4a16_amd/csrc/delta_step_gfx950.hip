// The gated delta rule token by token.
//
//   S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
// Both sums over the state come from one pass over the old one:
//   u = beta (v - e^g S^T k),  o = scale (e^g S^T q + (k . q) u),  S <- e^g S + k u^T
// A wave keeps sixteen columns of one head's state in registers: lane 4 r + c has rows
// Dk / 16 r .. of columns 4 c .. 4 c + 3, so that a token costs no barrier and its key and query
// one load in each lane.  Columns do not depend on each other.
// Bound by memory for one token (the state in and out, 2 x 4 Dk Dv bytes a head).  48 heads of 128 x
// 128: one sequence 5.5 us, 64 of them 66 to 87, 6.1 to 4.7 TB/s (the last level of cache holds some).

#include <type_traits>

#include "delta_device.hpp"

namespace w4a16 {
namespace {

constexpr int kColumns = 16;           // of a wave
constexpr int kWaves = 4;              // of a workgroup: whole lines of memory (64 sequences, states cached in part: 67 us, with one wave 95)

// What a lane needs of one token.
template <int ROWS>
struct Token {
    u2 q[ROWS / 4], k[ROWS / 4], v;
};

template <bool BF, int DK>
__global__ void __launch_bounds__(64 * kWaves) step_kernel(DeltaArgs a) {
    constexpr int kRows = DK / 16;
    const int lane = threadIdx.x & 63, r = lane >> 2;
    const int col = (blockIdx.x * kWaves + (threadIdx.x >> 6)) * kColumns + 4 * (lane & 3);
    const int h = blockIdx.y, hk = h / (a.v_heads / a.k_heads);
    Seq s;
    if (!seq_of(a.s, blockIdx.z, &s)) return;

    float *const state = a.state + ((max(s.state, (int64_t)0) * a.v_heads + h) * DK + kRows * r) * a.value_dim + col;
    f4 S[kRows];
    if (s.fresh) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i] = f4{0.f, 0.f, 0.f, 0.f};
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i] = *reinterpret_cast<const f4 *>(state + (int64_t)i * a.value_dim);
    }
    const uint16_t *const q0 = static_cast<const uint16_t *>(a.q) + hk * DK + kRows * r;
    const uint16_t *const k0 = static_cast<const uint16_t *>(a.k) + hk * DK + kRows * r;
    const uint16_t *const v0 = static_cast<const uint16_t *>(a.v) + h * a.value_dim + col;
    auto load = [&](int t) {
        const int64_t row = s.first + t;
        Token<kRows> x;
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
            x.q[i] = *reinterpret_cast<const u2 *>(q0 + row * a.q_stride + 4 * i);
            x.k[i] = *reinterpret_cast<const u2 *>(k0 + row * a.k_stride + 4 * i);
        }
        x.v = *reinterpret_cast<const u2 *>(v0 + row * a.v_stride);
        return x;
    };

    Token<kRows> next = load(0);
    const float rate = a.a_log ? expf(a.a_log[h]) : 0.f, bias = a.a_log ? a.dt_bias[h] : 0.f;
    float all_keep = 0.f, all_beta = 0.f;      // of 64 tokens, one in each lane
    for (int t = 0; t < s.n; ++t) {
        const Token<kRows> x = next;
        if (t + 1 < s.n) next = load(t + 1);
        if (t % 64 == 0) {
            const Gates gate = t + lane < s.n ? gates_of<BF>(a, s.first + t + lane, h, rate, bias) : Gates{0.f, 0.f};
            all_keep = expf(gate.g);
            all_beta = gate.beta;
        }
        const float keep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all_keep), t % 64));
        const float beta = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all_beta), t % 64));
        float q[kRows], k[kRows];
#pragma unroll
        for (int i = 0; i < kRows; i += 2) {
            q[i] = lo_f32<BF>(x.q[i / 4][i / 2 % 2]);
            q[i + 1] = hi_f32<BF>(x.q[i / 4][i / 2 % 2]);
            k[i] = lo_f32<BF>(x.k[i / 4][i / 2 % 2]);
            k[i + 1] = hi_f32<BF>(x.k[i / 4][i / 2 % 2]);
        }
        const f4 v = {lo_f32<BF>(x.v[0]), hi_f32<BF>(x.v[0]), lo_f32<BF>(x.v[1]), hi_f32<BF>(x.v[1])};
        if (a.unit) {
            to_unit<4>(k, a.eps);
            to_unit<4>(q, a.eps);
        }
        float qk = 0.f;
        f4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            qk = __builtin_fmaf(q[i], k[i], qk);
            sk += S[i] * k[i];
            sq += S[i] * q[i];
        }
        qk = over_lanes<4>(qk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] = over_lanes<4>(sk[e]);
            sq[e] = over_lanes<4>(sq[e]);
        }
        const f4 u = beta * (v - keep * sk);
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i] = keep * S[i] + k[i] * u;
        if (r == 0) {
            const f4 o = a.scale * (keep * sq + qk * u);
            *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + (s.first + t) * a.out_stride + (int64_t)h * a.value_dim + col) =
                pack4<BF>(o[0], o[1], o[2], o[3]);
        }
    }
    if (s.state < 0) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i) *reinterpret_cast<f4 *>(state + (int64_t)i * a.value_dim) = S[i];
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream) {
    const dim3 grid(a.value_dim / (kColumns * kWaves), a.v_heads, a.s.batch);
    auto go = [&](auto bf, auto dk) {
        step_kernel<bf(), dk()><<<grid, 64 * kWaves, 0, stream>>>(a);
        return hipGetLastError();
    };
    auto typed = [&](auto dk) { return a.bf16 ? go(std::true_type{}, dk) : go(std::false_type{}, dk); };
    return a.key_dim == 64 ? typed(std::integral_constant<int, 64>{}) : typed(std::integral_constant<int, 128>{});
}

}  // namespace w4a16
