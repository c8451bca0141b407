// Internal launch interface of the gated delta rule and the short convolution (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

// The sequences of a call and the pool of states that they continue.  A state index outside
// [0, num_states) is not there: it stands for zeros, and nothing is written.
struct Sequences {
    const int32_t *cu = nullptr;           // [batch + 1] rows of each sequence
    const int32_t *index = nullptr;        // [batch] its state
    const int32_t *seen = nullptr;         // [batch] tokens that the state holds (0: zeros), or null: some
    const int64_t *tree = nullptr;         // [T] what each token descends from, or null: tokens in a row
    int64_t T = 0;
    int batch = 0, max_q = 0, num_states = 0;
};

struct ConvArgs {
    Sequences s;
    const void *x = nullptr;               // [T, channels]
    int64_t x_stride = 0;
    const float *weight = nullptr;         // [channels, width]
    const float *bias = nullptr;           // [channels], or null
    void *state = nullptr;                 // [num_states, width - 1, channels]
    void *out = nullptr;                   // [T, channels]
    int64_t out_stride = 0;
    int channels = 0, width = 0;
    bool bf16 = false, silu = false;
};
// Workgroups (of conv_threads threads) of a launch, for the host's check of its limits.
int64_t conv_blocks(const ConvArgs &a);
int conv_threads(const ConvArgs &a);
hipError_t launch_short_conv(const ConvArgs &a, hipStream_t stream);

struct DeltaArgs {
    Sequences s;
    const void *q = nullptr, *k = nullptr, *v = nullptr;   // [T, heads, dim]
    int64_t q_stride = 0, k_stride = 0, v_stride = 0;
    const void *a = nullptr, *b = nullptr;                 // [T, v_heads]
    int64_t a_stride = 0, b_stride = 0;
    const float *a_log = nullptr, *dt_bias = nullptr;      // [v_heads], or null: a and b hold g and beta in fp32
    float *state = nullptr;                                // [num_states, v_heads, key_dim, value_dim]
    void *out = nullptr;                                   // [T, v_heads, value_dim]
    int64_t out_stride = 0;
    int k_heads = 0, v_heads = 0, key_dim = 0, value_dim = 0;
    float scale = 1.f, eps = 0.f;
    bool bf16 = false, unit = false;
    void *workspace = nullptr;
};
// Token by token, the state in registers, for a few tokens of each sequence (no tree).
hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream);
// 64 tokens at a time, or a tree.
size_t delta_chunk_workspace_bytes(const DeltaArgs &a);
hipError_t launch_delta_chunk(const DeltaArgs &a, hipStream_t stream);

}  // namespace w4a16
