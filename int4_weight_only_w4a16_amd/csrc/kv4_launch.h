// Internal launch interface of the 4-bit key/value cache kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace w4a16 {

// f(head_dim, groups) with both as compile-time constants, for every pair the
// cache takes (head_dim 64, 128 or 256 in groups of 32, 64 or 128 channels).
template <typename F>
hipError_t kv4_dispatch(int head_dim, int groups, F f) {
    using std::integral_constant;
    const int key = 16 * head_dim + groups;
    switch (key) {
#define W4A16_KV4_SHAPE(D, NG) \
    case 16 * D + NG: return f(integral_constant<int, D>{}, integral_constant<int, NG>{});
        W4A16_KV4_SHAPE(64, 1)
        W4A16_KV4_SHAPE(64, 2)
        W4A16_KV4_SHAPE(128, 1)
        W4A16_KV4_SHAPE(128, 2)
        W4A16_KV4_SHAPE(128, 4)
        W4A16_KV4_SHAPE(256, 2)
        W4A16_KV4_SHAPE(256, 4)
        W4A16_KV4_SHAPE(256, 8)
#undef W4A16_KV4_SHAPE
        default: return hipErrorInvalidValue;
    }
}

// The current device if it is a gfx950 (with its CU count and LDS limit), else -1.
int usable_device(int *num_cus, size_t *max_lds);

// A cache and the sequences in it, as the kernels see them.  Slots of
// sequence b beyond table_stride * page_size, or on a page id outside
// [0, num_pages), are not there: never read, never written.
struct Kv4Cache {
    uint8_t *pages = nullptr;          // [num_pages][kv_heads][tiles_per_page][tile bytes]
    const int32_t *table = nullptr;    // [batch][table_stride]
    int num_pages = 0, kv_heads = 0, tiles_per_page = 0, table_stride = 0, batch = 0;
    int head_dim = 0, groups = 0;      // groups = head_dim / group_size
    bool bf16 = false;                 // type of the parameters (and of q, k, v and the output)
};

// Norm and rotation of one set of heads: x [T, heads, D] with a row stride.
struct RopeArgs {
    const float *cos = nullptr, *sin = nullptr;    // [max_pos, rot / 2], or null: no rotation
    const int32_t *positions = nullptr;            // [T]
    int rot = 0, max_pos = 0;
    bool interleaved = false;
    float eps = 0.f;
};
struct HeadsArgs {
    const void *x = nullptr;
    int64_t x_stride = 0;      // elements between tokens
    void *y = nullptr;
    int64_t y_stride = 0;
    const float *weight = nullptr;     // [D], or null: no norm
    int heads = 0;
};

hipError_t launch_qk_norm_rope(const HeadsArgs &q, const HeadsArgs &k, const RopeArgs &r, int64_t T,
                               int head_dim, bool bf16, hipStream_t stream);

struct Kv4AppendArgs {
    Kv4Cache c;
    HeadsArgs q, k, v;                 // q.heads == 0: keys and values only; k.y, v.* beyond x unused
    RopeArgs r;
    const int32_t *cu = nullptr, *kv_len = nullptr;    // [batch + 1], [batch]
    int64_t T = 0;
    int max_q = 0;
};
hipError_t launch_kv4_append(const Kv4AppendArgs &a, hipStream_t stream);

struct Kv4ReadArgs {
    Kv4Cache c;
    const int32_t *cu = nullptr, *kv_len = nullptr;
    void *k = nullptr, *v = nullptr;   // [rows, kv_heads, D]
    int64_t rows = 0;
};
hipError_t launch_kv4_read(const Kv4ReadArgs &a, hipStream_t stream);

struct Kv4AttnArgs {
    Kv4Cache c;
    const void *q = nullptr;           // [T, q_heads, D]
    int64_t q_stride = 0;
    const int32_t *cu = nullptr, *kv_len = nullptr;
    void *out = nullptr;               // attention: [T, q_heads, D]
    int64_t out_stride = 0;
    float *lse = nullptr;              // [T, q_heads]: attention writes it (or null), mass reads it
    float *acc = nullptr;              // mass: [batch, kv_heads, acc_stride]
    int64_t acc_stride = 0;
    int64_t T = 0;
    int q_heads = 0, max_q = 0, max_kv = 0, window = 0;    // window 0: none
    bool causal = true;
    const int64_t *tree = nullptr;     // [T]: bit j: the token descends from new token j; or null
    float scale = 1.f;
    void *workspace = nullptr;
};
// Tiles of rows that a head of one sequence is divided into (the attention's launch has them and
// the heads in one dimension).
int64_t kv4_attention_row_tiles(const Kv4AttnArgs &a);
int64_t kv4_tree_blocks(const Kv4AttnArgs &a);       // in the first dimension of a tree's launch
size_t kv4_attention_workspace_bytes(const Kv4AttnArgs &a);
hipError_t launch_kv4_attention(const Kv4AttnArgs &a, hipStream_t stream);
hipError_t launch_kv4_mass(const Kv4AttnArgs &a, hipStream_t stream);

struct Kv4EvictArgs {
    Kv4Cache c;                        // source; the destination lies in the same pages
    const int32_t *dst_table = nullptr;    // [batch][dst_stride]
    int dst_stride = 0;
    const int32_t *kv_len = nullptr;
    const float *acc = nullptr;        // [batch, kv_heads, acc_stride]
    int64_t acc_stride = 0;
    int budget = 0, recent = 0, max_kv = 0;
    int32_t *kept = nullptr;           // [batch, kv_heads, budget]
    int32_t *new_len = nullptr;        // [batch]
    float *acc_out = nullptr;          // [batch, kv_heads, budget]
};
hipError_t launch_kv4_evict(const Kv4EvictArgs &a, hipStream_t stream);

}  // namespace w4a16
