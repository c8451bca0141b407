// C ABI of the 4-bit key/value cache: argument validation and launches.  See
// include/w4a16.h for the contract.  Every check runs before any HIP call.

#include <cmath>

#include "../../include/w4a16.h"
#include "kv4_launch.h"

namespace {

// Indices inside a tile, a table row or a launch are 32 bits; addresses of
// pages and of rows of q, k, v are 64 bits.
constexpr int64_t kMax = ((int64_t)1 << 31) - 1;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool in_range(int64_t v, int64_t lo, int64_t hi = kMax) { return v >= lo && v <= hi; }

int check_geometry(int64_t kv_heads, int64_t head_dim, int64_t group, int64_t page_size) {
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return W4A16_ERR_SHAPE;
    if (!in_range(kv_heads, 1, 1 << 15) || page_size < 32 || page_size % 32 != 0) return W4A16_ERR_SHAPE;
    if ((group != 32 && group != 64 && group != 128) || group > head_dim) return W4A16_ERR_GROUP;
    // group >= head_dim / 8 holds for all of them
    const int64_t tile = 32 * (head_dim + 8 * (head_dim / group));
    if (page_size > kMax || kv_heads * (page_size / 32) * tile > kMax) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

struct CacheShape {
    int64_t kv_heads, head_dim, group, page_size, num_pages, batch, table_stride;
};

int check_cache(const CacheShape &s) {
    const int st = check_geometry(s.kv_heads, s.head_dim, s.group, s.page_size);
    if (st != W4A16_OK) return st;
    if (!in_range(s.num_pages, 0) || !in_range(s.batch, 0, 65535) || !in_range(s.table_stride, 0) ||
        s.table_stride > kMax / s.page_size)
        return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

int check_cache_pointers(const void *pages, const int32_t *table, const int32_t *cu, const int32_t *kv_len) {
    if (!pages || !table || !cu || !kv_len) return W4A16_ERR_NULL;
    if (!aligned(pages, 16) || !aligned(table, 4) || !aligned(cu, 4) || !aligned(kv_len, 4))
        return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

w4a16::Kv4Cache make_cache(const void *pages, const int32_t *table, const CacheShape &s, unsigned flags) {
    w4a16::Kv4Cache c;
    c.pages = static_cast<uint8_t *>(const_cast<void *>(pages));
    c.table = table;
    c.num_pages = (int)s.num_pages;
    c.kv_heads = (int)s.kv_heads;
    c.tiles_per_page = (int)(s.page_size / 32);
    c.table_stride = (int)s.table_stride;
    c.batch = (int)s.batch;
    c.head_dim = (int)s.head_dim;
    c.groups = (int)(s.head_dim / s.group);
    c.bf16 = (flags & W4A16_X_BF16) != 0;
    return c;
}

// A token-major set of heads: [T, heads, D] with a row stride.
int check_stride(int64_t stride, int64_t heads, int64_t D, int64_t T) {
    if (stride % 8 != 0 || stride < heads * D || stride > kMax) return W4A16_ERR_SHAPE;
    return in_range(T, 0, 1 << 28) ? W4A16_OK : W4A16_ERR_SHAPE;
}

struct RopeIn {
    const float *cos, *sin;
    const int32_t *positions;
    int64_t rot_dim, max_pos;
    float eps;
};

int check_rope(const RopeIn &r, int64_t D) {
    if (!(r.eps >= 0.f) || !std::isfinite(r.eps)) return W4A16_ERR_SHAPE;
    if (!r.cos && !r.sin) return W4A16_OK;
    if (!r.cos || !r.sin || !r.positions) return W4A16_ERR_NULL;
    if (r.rot_dim < 16 || r.rot_dim % 16 != 0 || r.rot_dim > D || !in_range(r.max_pos, 1))
        return W4A16_ERR_SHAPE;
    if (!aligned(r.cos, 16) || !aligned(r.sin, 16) || !aligned(r.positions, 4)) return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

w4a16::RopeArgs make_rope(const RopeIn &r, unsigned flags) {
    w4a16::RopeArgs a;
    a.cos = r.cos;
    a.sin = r.sin;
    a.positions = r.positions;
    a.rot = r.cos ? (int)r.rot_dim : 0;
    a.max_pos = r.cos ? (int)r.max_pos : 0;
    a.interleaved = (flags & W4A16_ROPE_INTERLEAVED) != 0;
    a.eps = r.eps;
    return a;
}

w4a16::HeadsArgs make_heads(const void *x, int64_t x_stride, void *y, int64_t y_stride, const float *weight,
                            int64_t heads) {
    w4a16::HeadsArgs a;
    a.x = x;
    a.x_stride = x_stride;
    a.y = y;
    a.y_stride = y_stride;
    a.weight = weight;
    a.heads = (int)heads;
    return a;
}

// Queries: heads, strides and pointers.
int check_queries(const void *q, int64_t q_stride, const void *out, int64_t out_stride, int64_t heads,
                  int64_t kv_heads, int64_t D, int64_t T) {
    if (!in_range(heads, 1, 1 << 15) || heads % kv_heads != 0) return W4A16_ERR_SHAPE;
    int st = check_stride(q_stride, heads, D, T);
    if (st == W4A16_OK) st = check_stride(out_stride, heads, D, T);
    if (st != W4A16_OK) return st;
    if (T > 0 && (!q || !out)) return W4A16_ERR_NULL;
    return aligned(q, 16) && aligned(out, 16) ? W4A16_OK : W4A16_ERR_ALIGN;
}

// A launch of `blocks` workgroups of `threads` in one dimension: it counts threads in 32 bits.
bool grid_ok(int64_t blocks, int64_t threads) { return blocks * threads <= UINT32_MAX; }

// Workgroups for `rows` rows of heads, eight channels a lane (norm and rotation).
constexpr int64_t kRowThreads = 256;
int64_t row_blocks(int64_t rows, int64_t D) { return (rows * (D / 8) + kRowThreads - 1) / kRowThreads; }

int launched(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

int device_ok() {
    int num_cus = 0;
    size_t max_lds = 0;
    return w4a16::usable_device(&num_cus, &max_lds) < 0 ? W4A16_ERR_DEVICE : W4A16_OK;
}

int check_attention(const CacheShape &s, int64_t T, int64_t q_heads, int64_t max_q, int64_t max_kv, int64_t window,
                    float scale, unsigned flags) {
    if ((flags & ~(W4A16_X_BF16 | W4A16_NONCAUSAL)) != 0 || ((flags & W4A16_NONCAUSAL) && window != 0))
        return W4A16_ERR_FLAGS;
    const int st = check_cache(s);
    if (st != W4A16_OK) return st;
    if (!in_range(max_q, 0, 1 << 24) || !in_range(max_kv, 0, kMax - 64) || !in_range(window, 0, kMax / 2) ||
        !std::isfinite(scale) || !(scale > 0.f))
        return W4A16_ERR_SHAPE;
    // rows of one sequence and head
    if (!in_range(q_heads, 1, 1 << 15) || q_heads / s.kv_heads * max_q > kMax / 2) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace

extern "C" size_t w4a16_kv4_page_bytes(int64_t kv_heads, int64_t head_dim, int64_t group_size,
                                       int64_t page_size) {
    if (check_geometry(kv_heads, head_dim, group_size, page_size) != W4A16_OK) return 0;
    return (size_t)(kv_heads * (page_size / 32) * 32 * (head_dim + 8 * (head_dim / group_size)));
}

extern "C" int w4a16_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                  const float *q_weight, const float *k_weight, float eps, const float *cos,
                                  const float *sin, const int32_t *positions, void *q_out, int64_t q_out_stride,
                                  void *k_out, int64_t k_out_stride, int64_t T, int64_t q_heads, int64_t kv_heads,
                                  int64_t head_dim, int64_t rot_dim, int64_t max_pos, unsigned flags,
                                  void *stream) {
    if ((flags & ~(W4A16_X_BF16 | W4A16_ROPE_INTERLEAVED)) != 0) return W4A16_ERR_FLAGS;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return W4A16_ERR_SHAPE;
    if (!in_range(q_heads, 0, 1 << 15) || !in_range(kv_heads, 0, 1 << 15)) return W4A16_ERR_SHAPE;
    const int64_t strides[4] = {q_stride, q_out_stride, k_stride, k_out_stride};
    const void *pointers[4] = {q, q_out, k, k_out};
    for (int i = 0; i < 4; ++i) {
        const int64_t heads = i < 2 ? q_heads : kv_heads;
        if (heads == 0) continue;
        const int st = check_stride(strides[i], heads, head_dim, T);
        if (st != W4A16_OK) return st;
        if (T > 0 && !pointers[i]) return W4A16_ERR_NULL;
        if (!aligned(pointers[i], 16)) return W4A16_ERR_ALIGN;
    }
    if (!in_range(T, 0, 1 << 28) || !grid_ok(row_blocks(T * (q_heads + kv_heads), head_dim), kRowThreads))
        return W4A16_ERR_SHAPE;
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return W4A16_ERR_ALIGN;
    const RopeIn rope{cos, sin, positions, rot_dim, max_pos, eps};
    const int st = check_rope(rope, head_dim);
    if (st != W4A16_OK) return st;
    if (T == 0 || q_heads + kv_heads == 0) return W4A16_OK;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    return launched(w4a16::launch_qk_norm_rope(
        make_heads(q, q_stride, q_out, q_out_stride, q_weight, q_heads),
        make_heads(k, k_stride, k_out, k_out_stride, k_weight, kv_heads), make_rope(rope, flags), T, (int)head_dim,
        (flags & W4A16_X_BF16) != 0, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int w4a16_kv4_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                int64_t v_stride, const float *q_weight, const float *k_weight, float eps,
                                const float *cos, const float *sin, const int32_t *positions, void *q_out,
                                int64_t q_out_stride, void *pages, const int32_t *table, const int32_t *cu_seqlens,
                                const int32_t *kv_len, int64_t T, int64_t q_heads, int64_t kv_heads,
                                int64_t head_dim, int64_t rot_dim, int64_t max_pos, int64_t group_size,
                                int64_t page_size, int64_t num_pages, int64_t batch, int64_t table_stride,
                                int64_t max_q, unsigned flags, void *stream) {
    if ((flags & ~(W4A16_X_BF16 | W4A16_ROPE_INTERLEAVED)) != 0) return W4A16_ERR_FLAGS;
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    int st = check_cache(s);
    if (st == W4A16_OK) st = check_stride(k_stride, kv_heads, head_dim, T);
    if (st == W4A16_OK) st = check_stride(v_stride, kv_heads, head_dim, T);
    if (st != W4A16_OK) return st;
    if (!in_range(max_q, 0, 1 << 28) || q_heads < 0) return W4A16_ERR_SHAPE;
    if (q_heads > 0) st = check_queries(q, q_stride, q_out, q_out_stride, q_heads, kv_heads, head_dim, T);
    if (st != W4A16_OK) return st;
    const RopeIn rope{cos, sin, positions, rot_dim, max_pos, eps};
    st = check_rope(rope, head_dim);
    if (st != W4A16_OK) return st;
    max_q = max_q < T ? max_q : T;               // (no sequence has more)
    if (!grid_ok(batch * ((max_q + 62) / 32) * kv_heads + row_blocks(T * q_heads, head_dim), kRowThreads))
        return W4A16_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
        return W4A16_ERR_ALIGN;
    if (T == 0) return W4A16_OK;
    if (!k || !v) return W4A16_ERR_NULL;
    st = check_cache_pointers(pages, table, cu_seqlens, kv_len);
    if (st != W4A16_OK) return st;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    w4a16::Kv4AppendArgs a;
    a.c = make_cache(pages, table, s, flags);
    a.q = make_heads(q, q_stride, q_out, q_out_stride, q_weight, q_heads);
    a.k = make_heads(k, k_stride, nullptr, 0, k_weight, kv_heads);
    a.v = make_heads(v, v_stride, nullptr, 0, nullptr, kv_heads);
    a.r = make_rope(rope, flags);
    a.cu = cu_seqlens;
    a.kv_len = kv_len;
    a.T = T;
    a.max_q = (int)max_q;
    return launched(w4a16::launch_kv4_append(a, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int w4a16_kv4_read(const void *pages, const int32_t *table, const int32_t *cu_seqlens,
                              const int32_t *kv_len, void *k, void *v, int64_t rows, int64_t kv_heads,
                              int64_t head_dim, int64_t group_size, int64_t page_size, int64_t num_pages,
                              int64_t batch, int64_t table_stride, unsigned flags, void *stream) {
    if ((flags & ~W4A16_X_BF16) != 0) return W4A16_ERR_FLAGS;
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    int st = check_cache(s);
    if (st != W4A16_OK) return st;
    if (!in_range(rows, 0, kMax - 32) || !grid_ok((rows + 31) / 32, kRowThreads)) return W4A16_ERR_SHAPE;
    if (rows == 0) return W4A16_OK;
    if (!k || !v) return W4A16_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return W4A16_ERR_ALIGN;
    st = check_cache_pointers(pages, table, cu_seqlens, kv_len);
    if (st != W4A16_OK) return st;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    w4a16::Kv4ReadArgs a;
    a.c = make_cache(pages, table, s, flags);
    a.cu = cu_seqlens;
    a.kv_len = kv_len;
    a.k = k;
    a.v = v;
    a.rows = rows;
    return launched(w4a16::launch_kv4_read(a, reinterpret_cast<hipStream_t>(stream)));
}

static w4a16::Kv4AttnArgs attention_args(const w4a16::Kv4Cache &c, const void *q, int64_t q_stride,
                                         const int32_t *cu, const int32_t *kv_len, int64_t T, int64_t q_heads,
                                         int64_t max_q, int64_t max_kv, float scale, int64_t window,
                                         unsigned flags) {
    w4a16::Kv4AttnArgs a;
    a.c = c;
    a.q = q;
    a.q_stride = q_stride;
    a.cu = cu;
    a.kv_len = kv_len;
    a.T = T;
    a.q_heads = (int)q_heads;
    a.max_q = (int)max_q;
    a.max_kv = (int)max_kv;
    a.window = (int)window;
    a.causal = (flags & W4A16_NONCAUSAL) == 0;
    a.scale = scale;
    return a;
}

// The attention's launch: heads and tiles of rows in its second dimension.
static bool attention_fits(const w4a16::Kv4AttnArgs &a) {
    return a.c.kv_heads * w4a16::kv4_attention_row_tiles(a) <= 65535;
}

// Attention of tokens in a row, or with `is_tree` of a tree.
static int attend(const CacheShape &s, const void *q, int64_t q_stride, const void *pages, const int32_t *table,
                  const int32_t *cu_seqlens, const int32_t *kv_len, bool is_tree, const int64_t *tree, void *out,
                  int64_t out_stride, float *lse, int64_t T, int64_t q_heads, int64_t max_q, int64_t max_kv,
                  float scale, int64_t window, unsigned flags, void *workspace, size_t workspace_bytes,
                  void *stream) {
    const int64_t kv_heads = s.kv_heads, head_dim = s.head_dim, batch = s.batch;
    int st = check_attention(s, T, q_heads, max_q, max_kv, window, scale, flags);
    if (st == W4A16_OK && is_tree) {
        if (flags & W4A16_NONCAUSAL) return W4A16_ERR_FLAGS;
        // (a window that a path of drafts could leave is not taken)
        if (max_q > W4A16_TREE_MAX || (window > 0 && window < W4A16_TREE_MAX)) return W4A16_ERR_SHAPE;
    }
    if (st == W4A16_OK) st = check_queries(q, q_stride, out, out_stride, q_heads, kv_heads, head_dim, T);
    if (st != W4A16_OK) return st;
    w4a16::Kv4AttnArgs a = attention_args(make_cache(pages, table, s, flags), q, q_stride, cu_seqlens, kv_len, T,
                                          q_heads, max_q, max_kv, scale, window, flags);
    if (!attention_fits(a)) return W4A16_ERR_SHAPE;
    if (!aligned(lse, 4) || !aligned(tree, 8)) return W4A16_ERR_ALIGN;
    if (T == 0 || batch == 0 || max_q == 0) return W4A16_OK;
    if (is_tree && !grid_ok(w4a16::kv4_tree_blocks(a), 512)) return W4A16_ERR_SHAPE;
    if (is_tree && !tree) return W4A16_ERR_NULL;
    st = check_cache_pointers(pages, table, cu_seqlens, kv_len);
    if (st != W4A16_OK) return st;
    a.tree = tree;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.workspace = workspace;
    const size_t need = w4a16::kv4_attention_workspace_bytes(a);
    if (need > 0) {
        if (!workspace) return W4A16_ERR_NULL;
        if (!aligned(workspace, 16)) return W4A16_ERR_ALIGN;
        if (workspace_bytes < need) return W4A16_ERR_WORKSPACE;
    }
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    return launched(w4a16::launch_kv4_attention(a, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int w4a16_kv4_attention(const void *q, int64_t q_stride, const void *pages, const int32_t *table,
                                   const int32_t *cu_seqlens, const int32_t *kv_len, void *out, int64_t out_stride,
                                   float *lse, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                   int64_t group_size, int64_t page_size, int64_t num_pages, int64_t batch,
                                   int64_t table_stride, int64_t max_q, int64_t max_kv, float scale, int64_t window,
                                   unsigned flags, void *workspace, size_t workspace_bytes, void *stream) {
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    return attend(s, q, q_stride, pages, table, cu_seqlens, kv_len, false, nullptr, out, out_stride, lse, T, q_heads,
                  max_q, max_kv, scale, window, flags, workspace, workspace_bytes, stream);
}

extern "C" int w4a16_kv4_tree_attention(const void *q, int64_t q_stride, const void *pages, const int32_t *table,
                                        const int32_t *cu_seqlens, const int32_t *kv_len, const int64_t *tree,
                                        void *out, int64_t out_stride, float *lse, int64_t T, int64_t q_heads,
                                        int64_t kv_heads, int64_t head_dim, int64_t group_size, int64_t page_size,
                                        int64_t num_pages, int64_t batch, int64_t table_stride, int64_t max_q,
                                        int64_t max_kv, float scale, int64_t window, unsigned flags,
                                        void *workspace, size_t workspace_bytes, void *stream) {
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    return attend(s, q, q_stride, pages, table, cu_seqlens, kv_len, true, tree, out, out_stride, lse, T, q_heads,
                  max_q, max_kv, scale, window, flags, workspace, workspace_bytes, stream);
}

extern "C" size_t w4a16_kv4_attention_workspace_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads,
                                                      int64_t head_dim, int64_t max_q, int64_t max_kv,
                                                      int64_t window) {
    const CacheShape s{kv_heads, head_dim, 64, 32, 0, batch, 0};
    if (kv_heads <= 0 || check_attention(s, 0, q_heads, max_q, max_kv, window, 1.f, 0) != W4A16_OK ||
        q_heads % kv_heads != 0 || batch == 0 || max_q == 0)
        return 0;
    const w4a16::Kv4AttnArgs a = attention_args(make_cache(nullptr, nullptr, s, 0), nullptr, 0, nullptr, nullptr, 0,
                                                q_heads, max_q, max_kv, 1.f, window, 0);
    return attention_fits(a) ? w4a16::kv4_attention_workspace_bytes(a) : 0;
}

extern "C" int w4a16_kv4_attention_mass(const void *q, int64_t q_stride, const void *pages, const int32_t *table,
                                        const int32_t *cu_seqlens, const int32_t *kv_len, const float *lse,
                                        float *acc, int64_t acc_stride, int64_t T, int64_t q_heads,
                                        int64_t kv_heads, int64_t head_dim, int64_t group_size, int64_t page_size,
                                        int64_t num_pages, int64_t batch, int64_t table_stride, int64_t max_q,
                                        int64_t max_kv, float scale, int64_t window, unsigned flags, void *stream) {
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    int st = check_attention(s, T, q_heads, max_q, max_kv, window, scale, flags);
    if (st == W4A16_OK) st = check_queries(q, q_stride, q, q_stride, q_heads, kv_heads, head_dim, T);
    if (st != W4A16_OK) return st;
    // (many rows: 128 threads a tile, up to eight tiles a workgroup)
    if (acc_stride < max_kv || !grid_ok((max_kv + 255) / 256, 1024)) return W4A16_ERR_SHAPE;
    if (!aligned(lse, 4) || !aligned(acc, 4)) return W4A16_ERR_ALIGN;
    if (T == 0 || batch == 0 || max_q == 0 || max_kv == 0) return W4A16_OK;
    if (!lse || !acc) return W4A16_ERR_NULL;
    st = check_cache_pointers(pages, table, cu_seqlens, kv_len);
    if (st != W4A16_OK) return st;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    w4a16::Kv4AttnArgs a = attention_args(make_cache(pages, table, s, flags), q, q_stride, cu_seqlens, kv_len, T,
                                          q_heads, max_q, max_kv, scale, window, flags);
    a.lse = const_cast<float *>(lse);
    a.acc = acc;
    a.acc_stride = acc_stride;
    return launched(w4a16::launch_kv4_mass(a, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int w4a16_kv4_evict(void *pages, const int32_t *table, const int32_t *kv_len, const float *acc,
                               int64_t acc_stride, int64_t budget, int64_t recent, const int32_t *dst_table,
                               int64_t dst_stride, int32_t *kept, int32_t *new_len, float *acc_out,
                               int64_t kv_heads, int64_t head_dim, int64_t group_size, int64_t page_size,
                               int64_t num_pages, int64_t batch, int64_t table_stride, int64_t max_kv,
                               unsigned flags, void *stream) {
    if ((flags & ~W4A16_X_BF16) != 0) return W4A16_ERR_FLAGS;
    const CacheShape s{kv_heads, head_dim, group_size, page_size, num_pages, batch, table_stride};
    int st = check_cache(s);
    if (st != W4A16_OK) return st;
    if (!in_range(budget, 1, kMax - 64) || recent < 0 || recent > budget || !in_range(max_kv, 0, kMax - 64) ||
        acc_stride < max_kv || !in_range(dst_stride, 1, kMax / page_size) || dst_stride * page_size < budget ||
        !grid_ok((budget + 31) / 32, 256))
        return W4A16_ERR_SHAPE;
    if (batch == 0) return W4A16_OK;
    st = check_cache_pointers(pages, table, kv_len, kv_len);
    if (st != W4A16_OK) return st;
    if ((!acc && max_kv > 0) || !dst_table || !kept || !new_len || !acc_out) return W4A16_ERR_NULL;
    if (!aligned(acc, 4) || !aligned(dst_table, 4) || !aligned(kept, 4) || !aligned(new_len, 4) ||
        !aligned(acc_out, 4))
        return W4A16_ERR_ALIGN;
    if (device_ok() != W4A16_OK) return W4A16_ERR_DEVICE;
    w4a16::Kv4EvictArgs a;
    a.c = make_cache(pages, table, s, flags);
    a.dst_table = dst_table;
    a.dst_stride = (int)dst_stride;
    a.kv_len = kv_len;
    a.acc = acc;
    a.acc_stride = acc_stride;
    a.budget = (int)budget;
    a.recent = (int)recent;
    a.max_kv = (int)max_kv;
    a.kept = kept;
    a.new_len = new_len;
    a.acc_out = acc_out;
    return launched(w4a16::launch_kv4_evict(a, reinterpret_cast<hipStream_t>(stream)));
}
