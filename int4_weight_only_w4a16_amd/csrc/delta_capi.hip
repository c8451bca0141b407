// C ABI of the short convolution and the gated delta rule: argument validation and launches.
// See include/w4a16.h for the contract.  Every check runs before any HIP call.

#include <algorithm>
#include <cmath>

#include "../../include/w4a16.h"
#include "delta_launch.h"
#include "kv4_launch.h"

namespace {

constexpr int64_t kMax = ((int64_t)1 << 31) - 1;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool in_range(int64_t v, int64_t lo, int64_t hi = kMax) { return v >= lo && v <= hi; }
int launched(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }
int device_ok() {
    int num_cus = 0;
    size_t max_lds = 0;
    return w4a16::usable_device(&num_cus, &max_lds) < 0 ? W4A16_ERR_DEVICE : W4A16_OK;
}

// A launch counts threads in 32 bits.
bool grid_ok(int64_t blocks, int64_t threads) { return blocks <= UINT32_MAX / threads; }

int check_sizes(int64_t T, int64_t batch, int64_t max_q, int64_t num_states, bool tree) {
    if (!in_range(T, 0, 1 << 28) || !in_range(batch, 0, 65535) || !in_range(max_q, 0, 1 << 28) ||
        !in_range(num_states, 0) || (tree && max_q > W4A16_TREE_MAX))
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int check_stride(int64_t stride, int64_t width) {
    return stride % 8 == 0 && stride >= width && stride <= kMax ? W4A16_OK : W4A16_ERR_SHAPE;
}

int check_sequences(const int32_t *index, const int32_t *seen, const int32_t *cu, const int64_t *tree) {
    if (!index || !cu) return W4A16_ERR_NULL;
    return aligned(index, 4) && aligned(seen, 4) && aligned(cu, 4) && aligned(tree, 8) ? W4A16_OK : W4A16_ERR_ALIGN;
}

w4a16::Sequences make_sequences(const int32_t *index, const int32_t *seen, const int32_t *cu, const int64_t *tree,
                                int64_t T, int64_t batch, int64_t max_q, int64_t num_states) {
    w4a16::Sequences s;
    s.cu = cu;
    s.index = index;
    s.seen = seen;
    s.tree = tree;
    s.T = T;
    s.batch = (int)batch;
    s.max_q = (int)(max_q < T ? max_q : T);      // (no sequence has more)
    s.num_states = (int)num_states;
    return s;
}

}  // namespace

extern "C" int w4a16_short_conv(const void *x, int64_t x_stride, const float *weight, const float *bias, void *state,
                                const int32_t *state_index, const int32_t *seen, const int32_t *cu_seqlens,
                                const int64_t *tree, void *out, int64_t out_stride, int64_t T, int64_t channels,
                                int64_t width, int64_t num_states, int64_t batch, int64_t max_q, unsigned flags,
                                void *stream) {
    if ((flags & ~(W4A16_X_BF16 | W4A16_SILU)) != 0) return W4A16_ERR_FLAGS;
    if (!in_range(channels, 8, 1 << 24) || channels % 8 != 0 || !in_range(width, 2, 4)) return W4A16_ERR_SHAPE;
    int st = check_sizes(T, batch, max_q, num_states, tree != nullptr);
    if (st == W4A16_OK) st = check_stride(x_stride, channels);
    if (st == W4A16_OK) st = check_stride(out_stride, channels);
    if (st != W4A16_OK) return st;
    w4a16::ConvArgs a;
    a.s = make_sequences(state_index, seen, cu_seqlens, tree, T, batch, max_q, num_states);
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    a.out = out;
    a.out_stride = out_stride;
    a.channels = (int)channels;
    a.width = (int)width;
    a.bf16 = (flags & W4A16_X_BF16) != 0;
    a.silu = (flags & W4A16_SILU) != 0;
    if (a.s.max_q > 0 && !grid_ok(w4a16::conv_blocks(a), w4a16::conv_threads(a))) return W4A16_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(state, 16) || !aligned(out, 16))
        return W4A16_ERR_ALIGN;
    if (T == 0 || batch == 0 || max_q == 0) return W4A16_OK;
    if (!x || !weight || !out || (!state && num_states > 0)) return W4A16_ERR_NULL;
    st = check_sequences(state_index, seen, cu_seqlens, tree);
    if (st != W4A16_OK) return st;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    return launched(w4a16::launch_short_conv(a, reinterpret_cast<hipStream_t>(stream)));
}

// Most tokens of a sequence that go token by token.  In steps and in chunks, us, 48 heads of 128 x 128
// (32 of 64 x 128):
//   tokens              8                 16                24
//   1 sequence      11 (9) and 17 (14)  18 (14) and 17 (15)   24 (20) and 17 (14)
//   8               22 (13) and 40 (24) 37 (21) and 40 (25)   51 (28) and 40 (25)
//   32              63 (34) and 104 (58) 111 (61) and 105 (58) 159 (86) and 107 (59)
static constexpr int64_t kStepTokens = 16;

static bool in_chunks(const w4a16::DeltaArgs &d) { return d.s.tree || d.s.max_q > kStepTokens; }

static int check_delta(int64_t T, int64_t k_heads, int64_t v_heads, int64_t key_dim, int64_t value_dim,
                       int64_t num_states, int64_t batch, int64_t max_q, bool tree) {
    if ((key_dim != 64 && key_dim != 128) || !in_range(value_dim, 64, 256) || value_dim % 64 != 0 ||
        !in_range(k_heads, 1, 1 << 12) || !in_range(v_heads, 1, 1 << 12) || v_heads % k_heads != 0)
        return W4A16_ERR_SHAPE;
    return check_sizes(T, batch, max_q, num_states, tree);
}

extern "C" int w4a16_delta_rule(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                int64_t v_stride, const void *a, int64_t a_stride, const void *b, int64_t b_stride,
                                const float *a_log, const float *dt_bias, float *state, const int32_t *state_index,
                                const int32_t *seen, const int32_t *cu_seqlens, const int64_t *tree, void *out,
                                int64_t out_stride, int64_t T, int64_t k_heads, int64_t v_heads, int64_t key_dim,
                                int64_t value_dim, int64_t num_states, int64_t batch, int64_t max_q, float scale,
                                float eps, unsigned flags, void *workspace, size_t workspace_bytes, void *stream) {
    if ((flags & ~(W4A16_X_BF16 | W4A16_UNIT_QK)) != 0) return W4A16_ERR_FLAGS;
    int st = check_delta(T, k_heads, v_heads, key_dim, value_dim, num_states, batch, max_q, tree != nullptr);
    if (st == W4A16_OK) st = check_stride(q_stride, k_heads * key_dim);
    if (st == W4A16_OK) st = check_stride(k_stride, k_heads * key_dim);
    if (st == W4A16_OK) st = check_stride(v_stride, v_heads * value_dim);
    if (st == W4A16_OK) st = check_stride(out_stride, v_heads * value_dim);
    if (st != W4A16_OK) return st;
    // (a chunk's rows are reached by 32-bit offsets)
    if (v_stride >= 1 << 23 || out_stride >= 1 << 23) return W4A16_ERR_SHAPE;
    if (!in_range(a_stride, v_heads) || !in_range(b_stride, v_heads) || !std::isfinite(scale) || !(scale > 0.f) ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return W4A16_ERR_SHAPE;
    const int gate_bytes = a_log ? 2 : 4;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(state, 16) ||
        !aligned(a, gate_bytes) || !aligned(b, gate_bytes) || !aligned(a_log, 4) || !aligned(dt_bias, 4))
        return W4A16_ERR_ALIGN;
    if ((a_log == nullptr) != (dt_bias == nullptr)) return W4A16_ERR_NULL;
    if (T == 0 || batch == 0 || max_q == 0) return W4A16_OK;
    if (!q || !k || !v || !a || !b || !out || (!state && num_states > 0)) return W4A16_ERR_NULL;
    st = check_sequences(state_index, seen, cu_seqlens, tree);
    if (st != W4A16_OK) return st;
    w4a16::DeltaArgs d;
    d.s = make_sequences(state_index, seen, cu_seqlens, tree, T, batch, max_q, num_states);
    d.q = q;
    d.q_stride = q_stride;
    d.k = k;
    d.k_stride = k_stride;
    d.v = v;
    d.v_stride = v_stride;
    d.a = a;
    d.a_stride = a_stride;
    d.b = b;
    d.b_stride = b_stride;
    d.a_log = a_log;
    d.dt_bias = dt_bias;
    d.state = state;
    d.out = out;
    d.out_stride = out_stride;
    d.k_heads = (int)k_heads;
    d.v_heads = (int)v_heads;
    d.key_dim = (int)key_dim;
    d.value_dim = (int)value_dim;
    d.scale = scale;
    d.eps = eps;
    d.bf16 = (flags & W4A16_X_BF16) != 0;
    d.unit = (flags & W4A16_UNIT_QK) != 0;
    d.workspace = workspace;
    const size_t need = in_chunks(d) ? w4a16::delta_chunk_workspace_bytes(d) : 0;
    if (need > 0) {
        if (!workspace) return W4A16_ERR_NULL;
        if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
        if (workspace_bytes < need) return W4A16_ERR_WORKSPACE;
    }
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    const hipStream_t on = reinterpret_cast<hipStream_t>(stream);
    return launched(in_chunks(d) ? w4a16::launch_delta_chunk(d, on) : w4a16::launch_delta_step(d, on));
}

extern "C" size_t w4a16_delta_rule_workspace_bytes(int64_t batch, int64_t T, int64_t k_heads, int64_t v_heads,
                                                   int64_t key_dim, int64_t value_dim, int64_t max_q, int tree) {
    if (check_delta(T, k_heads, v_heads, key_dim, value_dim, 0, batch, max_q, tree != 0) != W4A16_OK || T == 0 ||
        batch == 0 || max_q == 0)
        return 0;
    static const int64_t some = 0;
    w4a16::DeltaArgs d;
    d.s = make_sequences(nullptr, nullptr, nullptr, tree ? &some : nullptr, T, batch, max_q, 0);
    d.k_heads = (int)k_heads;
    d.v_heads = (int)v_heads;
    d.key_dim = (int)key_dim;
    d.value_dim = (int)value_dim;
    size_t most = 0;                   // over both types: what a call is cut into depends on its own
    for (const bool bf16 : {false, true}) {
        d.bf16 = bf16;
        if (in_chunks(d)) most = std::max(most, w4a16::delta_chunk_workspace_bytes(d));
    }
    return most;
}
