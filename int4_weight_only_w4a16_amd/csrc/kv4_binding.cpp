// Python binding of the 4-bit key/value cache's entry points: argument checks,
// outputs and workspaces from torch, and the C ABI call of include/w4a16.h.
//
// These calls run once for each layer and token, where a decode step is bound
// by how fast launches are issued: in C++ a call costs a few microseconds less
// than the kernel it launches takes, through ctypes three to five times that.

#include "binding.hpp"

namespace {

using namespace binding;

struct Geometry {
    int64_t heads, group, page, pages;
};

Geometry geometry_of(const Tensor &pages, int64_t D) {
    if (pages.dim() != 4 || pages.scalar_type() != at::kByte || !pages.is_cuda() || !pages.is_contiguous())
        refuse("pages must be a contiguous uint8 device tensor [pages, kv_heads, page_size / 32, tile bytes]");
    const int64_t tile = pages.size(3), groups = (tile / 32 - D) / 8;
    if (groups < 1 || D % groups != 0 || tile != 32 * (D + 8 * groups))
        refuse("pages with tiles of " + std::to_string(tile) + " bytes do not hold heads of " + std::to_string(D) +
               " channels");
    return {pages.size(1), D / groups, 32 * pages.size(2), pages.size(0)};
}

struct Sequences {
    int64_t batch, stride;
    const int32_t *table, *cu, *kv_len;
};

Sequences sequences_of(const Tensor &pages, const Tensor &table, const Tensor *cu, const Tensor &kv_len) {
    if (table.dim() != 2) refuse("block_table must be [batch, pages]");
    Sequences s{table.size(0), table.size(1), nullptr, nullptr, nullptr};
    s.table = static_cast<int32_t *>(plain("block_table", table, at::kInt, pages.device()));
    s.kv_len = static_cast<int32_t *>(plain("kv_len", kv_len, at::kInt, pages.device(), {s.batch}));
    if (cu) s.cu = static_cast<int32_t *>(plain("cu_seqlens", *cu, at::kInt, pages.device(), {s.batch + 1}));
    return s;
}

struct Rope {
    const float *q_weight = nullptr, *k_weight = nullptr, *cos = nullptr, *sin = nullptr;
    const int32_t *positions = nullptr;
    int64_t rot = 0, max_pos = 0;
};

Rope rope_of(const MaybeTensor &q_weight, const MaybeTensor &k_weight, const MaybeTensor &cos, const MaybeTensor &sin,
             const MaybeTensor &positions, int64_t D, int64_t T, const at::Device &device) {
    Rope r;
    if (q_weight) r.q_weight = static_cast<float *>(plain("norm weight", *q_weight, at::kFloat, device, {D}));
    if (k_weight) r.k_weight = static_cast<float *>(plain("norm weight", *k_weight, at::kFloat, device, {D}));
    if (cos.has_value() != sin.has_value() || cos.has_value() != positions.has_value())
        refuse("cos, sin and positions go together");
    if (cos) {
        if (cos->dim() != 2) refuse("cos and sin must be [positions, rot_dim / 2]");
        r.cos = static_cast<float *>(plain("cos", *cos, at::kFloat, device));
        r.sin = static_cast<float *>(plain("sin", *sin, at::kFloat, device, {cos->size(0), cos->size(1)}));
        r.positions = static_cast<int32_t *>(plain("positions", *positions, at::kInt, device, {T}));
        r.rot = 2 * cos->size(1);
        r.max_pos = cos->size(0);
    }
    return r;
}

Tensor output(const MaybeTensor &t, const Tensor &like) {
    if (!t) return at::empty(like.sizes(), like.options());
    if (t->sizes() != like.sizes()) refuse("an output must have the shape of its input");
    return *t;
}

std::tuple<Tensor, Tensor> qk_norm_rope(const Tensor &q, const Tensor &k, const MaybeTensor &q_weight,
                                        const MaybeTensor &k_weight, const MaybeTensor &cos, const MaybeTensor &sin,
                                        const MaybeTensor &positions, double eps, bool interleaved,
                                        const MaybeTensor &q_out, const MaybeTensor &k_out,
                                        const py::object &stream) {
    const int64_t qs = heads_stride("q", q), ks = heads_stride("k", k, &q);
    const int64_t T = q.size(0), D = q.size(2);
    if (k.size(0) != T || k.size(2) != D) refuse("q and k must have the same tokens and channels");
    const unsigned flags = type_flag(q.scalar_type()) | (interleaved ? W4A16_ROPE_INTERLEAVED : 0);
    const Rope r = rope_of(q_weight, k_weight, cos, sin, positions, D, T, q.device());
    const On on(q, stream);
    const Tensor qo = output(q_out, q), ko = output(k_out, k);
    check(w4a16_qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks, r.q_weight, r.k_weight, (float)eps, r.cos, r.sin,
                             r.positions, qo.data_ptr(), heads_stride("q_out", qo, &q), ko.data_ptr(),
                             heads_stride("k_out", ko, &q), T, q.size(1), k.size(1), D, r.rot, r.max_pos, flags,
                             on.stream()),
          "w4a16_qk_norm_rope");
    return {qo, ko};
}

MaybeTensor kv4_append(const Tensor &pages, const Tensor &k, const Tensor &v, const Tensor &block_table,
                       const Tensor &cu_seqlens, const Tensor &kv_len, int64_t max_q, const MaybeTensor &q,
                       const MaybeTensor &q_weight, const MaybeTensor &k_weight, const MaybeTensor &cos,
                       const MaybeTensor &sin, const MaybeTensor &positions, double eps, bool interleaved,
                       const MaybeTensor &q_out, const py::object &stream) {
    const int64_t ks = heads_stride("k", k), vs = heads_stride("v", v, &k);
    const int64_t T = k.size(0), hk = k.size(1), D = k.size(2);
    const Geometry g = geometry_of(pages, D);
    if (v.sizes() != k.sizes() || hk != g.heads || k.device() != pages.device())
        refuse("k and v must be [tokens, kv_heads, channels] of the cache, on its device");
    const Sequences s = sequences_of(pages, block_table, &cu_seqlens, kv_len);
    const unsigned flags = type_flag(k.scalar_type()) | (interleaved ? W4A16_ROPE_INTERLEAVED : 0);
    const Rope r = rope_of(q_weight, k_weight, cos, sin, positions, D, T, k.device());
    const On on(k, stream);
    MaybeTensor qo;
    int64_t qs = 0, qos = 0, hq = 0;
    if (q) {
        qs = heads_stride("q", *q, &k);
        hq = q->size(1);
        if (q->size(0) != T || q->size(2) != D) refuse("q must have the tokens and channels of k");
        qo = output(q_out, *q);
        qos = heads_stride("q_out", *qo, &k);
    } else if (q_out) {
        refuse("q_out without q");
    }
    check(w4a16_kv4_append(q ? q->data_ptr() : nullptr, qs, k.data_ptr(), ks, v.data_ptr(), vs, r.q_weight,
                           r.k_weight, (float)eps, r.cos, r.sin, r.positions, qo ? qo->data_ptr() : nullptr, qos,
                           pages.data_ptr(), s.table, s.cu, s.kv_len, T, hq, hk, D, r.rot, r.max_pos, g.group,
                           g.page, g.pages, s.batch, s.stride, max_q, flags, on.stream()),
          "w4a16_kv4_append");
    return qo;
}

std::tuple<Tensor, Tensor> kv4_read(const Tensor &pages, const Tensor &block_table, const Tensor &cu_seqlens,
                                    const Tensor &kv_len, int64_t rows, int64_t head_dim, at::ScalarType dtype,
                                    const MaybeTensor &k_out, const MaybeTensor &v_out, const py::object &stream) {
    const Geometry g = geometry_of(pages, head_dim);
    const Sequences s = sequences_of(pages, block_table, &cu_seqlens, kv_len);
    const unsigned flags = type_flag(dtype);
    if (rows < 0) refuse("rows must not be negative");
    const On on(pages, stream);
    Tensor out[2];
    void *ptr[2];
    for (int i = 0; i < 2; ++i) {
        const MaybeTensor &t = i ? v_out : k_out;
        out[i] = t ? *t : at::empty({rows, g.heads, head_dim}, pages.options().dtype(dtype));
        ptr[i] = plain("an output", out[i], dtype, pages.device(), {rows, g.heads, head_dim});
    }
    check(w4a16_kv4_read(pages.data_ptr(), s.table, s.cu, s.kv_len, ptr[0], ptr[1], rows, g.heads, head_dim, g.group,
                         g.page, g.pages, s.batch, s.stride, flags, on.stream()),
          "w4a16_kv4_read");
    return {out[0], out[1]};
}

Geometry attention_geometry(const Tensor &q, const Tensor &pages) {
    const Geometry g = geometry_of(pages, q.size(2));
    if (g.heads == 0 || q.size(1) % g.heads != 0 || q.device() != pages.device())
        refuse("q must be on the cache's device with a multiple of its heads");
    return g;
}

float scale_of(std::optional<double> scale, int64_t D) {
    return (float)(scale ? *scale : 1.0 / std::sqrt((double)D));
}

// Attention of tokens in a row, or of a tree.
py::object attend(const Tensor &q, const Tensor &pages, const Tensor &block_table, const Tensor &cu_seqlens,
                  const Tensor &kv_len, const Tensor *tree, int64_t max_q, int64_t max_kv,
                  std::optional<double> scale, bool causal, int64_t window, const MaybeTensor &out, bool return_lse,
                  const MaybeTensor &lse, const MaybeTensor &workspace, const py::object &stream) {
    const int64_t qs = heads_stride("q", q);
    const Geometry g = attention_geometry(q, pages);
    const Sequences s = sequences_of(pages, block_table, &cu_seqlens, kv_len);
    const int64_t T = q.size(0), hq = q.size(1), D = q.size(2);
    const unsigned flags = type_flag(q.scalar_type()) | (causal ? 0 : W4A16_NONCAUSAL);
    const On on(q, stream);
    const Tensor o = output(out, q);
    MaybeTensor l = lse;
    if (!l && return_lse) l = at::empty({T, hq}, q.options().dtype(at::kFloat));
    float *lse_ptr = l ? static_cast<float *>(plain("lse", *l, at::kFloat, q.device(), {T, hq})) : nullptr;
    const size_t need = w4a16_kv4_attention_workspace_bytes(s.batch, hq, g.heads, D, max_q, max_kv, window);
    Tensor ws;
    if (workspace) {
        ws = *workspace;
        plain("workspace", ws, ws.scalar_type(), pages.device());     // (any type: bytes are what counts)
    } else if (need)
        ws = at::empty({(int64_t)need}, pages.options());
    const int64_t os = heads_stride("out", o, &q);
    void *ws_ptr = ws.defined() ? ws.data_ptr() : nullptr;
    const size_t ws_bytes = ws.defined() ? ws.nbytes() : 0;
    if (tree) {
        const auto *words = static_cast<int64_t *>(plain("tree", *tree, at::kLong, q.device(), {T}));
        check(w4a16_kv4_tree_attention(q.data_ptr(), qs, pages.data_ptr(), s.table, s.cu, s.kv_len, words,
                                       o.data_ptr(), os, lse_ptr, T, hq, g.heads, D, g.group, g.page, g.pages,
                                       s.batch, s.stride, max_q, max_kv, scale_of(scale, D), window, flags, ws_ptr,
                                       ws_bytes, on.stream()),
              "w4a16_kv4_tree_attention");
    } else {
        check(w4a16_kv4_attention(q.data_ptr(), qs, pages.data_ptr(), s.table, s.cu, s.kv_len, o.data_ptr(), os,
                                  lse_ptr, T, hq, g.heads, D, g.group, g.page, g.pages, s.batch, s.stride, max_q,
                                  max_kv, scale_of(scale, D), window, flags, ws_ptr, ws_bytes, on.stream()),
              "w4a16_kv4_attention");
    }
    return return_lse ? py::cast(std::make_tuple(o, *l)) : py::cast(o);
}

py::object kv4_attention(const Tensor &q, const Tensor &pages, const Tensor &block_table, const Tensor &cu_seqlens,
                         const Tensor &kv_len, int64_t max_q, int64_t max_kv, std::optional<double> scale,
                         bool causal, int64_t window, const MaybeTensor &out, bool return_lse,
                         const MaybeTensor &lse, const MaybeTensor &workspace, const py::object &stream) {
    return attend(q, pages, block_table, cu_seqlens, kv_len, nullptr, max_q, max_kv, scale, causal, window, out,
                  return_lse, lse, workspace, stream);
}

py::object kv4_tree_attention(const Tensor &q, const Tensor &pages, const Tensor &block_table,
                              const Tensor &cu_seqlens, const Tensor &kv_len, const Tensor &tree, int64_t max_q,
                              int64_t max_kv, std::optional<double> scale, int64_t window, const MaybeTensor &out,
                              bool return_lse, const MaybeTensor &lse, const MaybeTensor &workspace,
                              const py::object &stream) {
    return attend(q, pages, block_table, cu_seqlens, kv_len, &tree, max_q, max_kv, scale, true, window, out,
                  return_lse, lse, workspace, stream);
}

float *weights_of(const Tensor &acc, const at::Device &device, int64_t batch, int64_t heads) {
    float *p = static_cast<float *>(plain("acc", acc, at::kFloat, device));
    if (acc.dim() != 3 || acc.size(0) != batch || acc.size(1) != heads) refuse("acc must be [batch, kv_heads, slots]");
    return p;
}

Tensor kv4_attention_mass(const Tensor &q, const Tensor &pages, const Tensor &block_table, const Tensor &cu_seqlens,
                          const Tensor &kv_len, const Tensor &lse, const Tensor &acc, int64_t max_q, int64_t max_kv,
                          std::optional<double> scale, bool causal, int64_t window, const py::object &stream) {
    const int64_t qs = heads_stride("q", q);
    const Geometry g = attention_geometry(q, pages);
    const Sequences s = sequences_of(pages, block_table, &cu_seqlens, kv_len);
    const int64_t T = q.size(0), hq = q.size(1), D = q.size(2);
    const unsigned flags = type_flag(q.scalar_type()) | (causal ? 0 : W4A16_NONCAUSAL);
    const float *lse_ptr = static_cast<float *>(plain("lse", lse, at::kFloat, q.device(), {T, hq}));
    float *acc_ptr = weights_of(acc, q.device(), s.batch, g.heads);
    const On on(q, stream);
    check(w4a16_kv4_attention_mass(q.data_ptr(), qs, pages.data_ptr(), s.table, s.cu, s.kv_len, lse_ptr, acc_ptr,
                                   acc.size(2), T, hq, g.heads, D, g.group, g.page, g.pages, s.batch, s.stride,
                                   max_q, max_kv, scale_of(scale, D), window, flags, on.stream()),
          "w4a16_kv4_attention_mass");
    return acc;
}

std::tuple<Tensor, Tensor, Tensor> kv4_evict(const Tensor &pages, const Tensor &block_table, const Tensor &kv_len,
                                             const Tensor &acc, int64_t budget, int64_t recent,
                                             const Tensor &dst_table, int64_t head_dim, int64_t max_kv,
                                             const py::object &stream) {
    const Geometry g = geometry_of(pages, head_dim);
    const Sequences s = sequences_of(pages, block_table, nullptr, kv_len);
    const float *acc_ptr = weights_of(acc, pages.device(), s.batch, g.heads);
    const auto *dst = static_cast<int32_t *>(plain("dst_table", dst_table, at::kInt, pages.device()));
    if (dst_table.dim() != 2 || dst_table.size(0) != s.batch) refuse("dst_table must be [batch, pages]");
    if (budget < 1) refuse("budget must be positive");
    const On on(pages, stream);
    const auto ints = pages.options().dtype(at::kInt);
    const Tensor kept = at::empty({s.batch, g.heads, budget}, ints), new_len = at::empty({s.batch}, ints);
    const Tensor acc_out = at::empty({s.batch, g.heads, budget}, pages.options().dtype(at::kFloat));
    check(w4a16_kv4_evict(pages.data_ptr(), s.table, s.kv_len, acc_ptr, acc.size(2), budget, recent, dst,
                          dst_table.size(1), static_cast<int32_t *>(kept.data_ptr()),
                          static_cast<int32_t *>(new_len.data_ptr()), static_cast<float *>(acc_out.data_ptr()),
                          g.heads, head_dim, g.group, g.page, g.pages, s.batch, s.stride, max_kv, 0, on.stream()),
          "w4a16_kv4_evict");
    return {kept, new_len, acc_out};
}

}  // namespace

void bind_delta(py::module_ &m);      // delta_binding.cpp

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    const auto none = py::none();
    bind_delta(m);
    m.def("qk_norm_rope", &qk_norm_rope, py::arg("q"), py::arg("k"), py::arg("q_weight") = none,
          py::arg("k_weight") = none, py::arg("cos") = none, py::arg("sin") = none, py::arg("positions") = none,
          py::arg("eps") = 1e-6, py::arg("interleaved") = false, py::arg("q_out") = none, py::arg("k_out") = none,
          py::arg("stream") = none,
          "RMS norm of each head of q [T, q_heads, D] and k [T, kv_heads, D] (weights fp32 [D], None: no norm),\n"
          "then the rotation of the first rot_dim channels by cos and sin (fp32 [positions, rot_dim / 2], None: no\n"
          "rotation) at positions (int32 [T]); pairs are (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved.\n"
          "Returns q_out and k_out (allocated unless given; they may be q and k themselves).");
    m.def("kv4_append", &kv4_append, py::arg("pages"), py::arg("k"), py::arg("v"), py::arg("block_table"),
          py::arg("cu_seqlens"), py::arg("kv_len"), py::arg("max_q"), py::arg("q") = none,
          py::arg("q_weight") = none, py::arg("k_weight") = none, py::arg("cos") = none, py::arg("sin") = none,
          py::arg("positions") = none, py::arg("eps") = 1e-6, py::arg("interleaved") = false,
          py::arg("q_out") = none, py::arg("stream") = none,
          "Quantise this call's keys and values [T, kv_heads, D] into the cache's last slots (kv_len counts them\n"
          "already); keys, and queries q [T, q_heads, D] if given, go through the norm and rotation of\n"
          "qk_norm_rope first, in the same launch.  max_q: at least the most tokens of any sequence.  Returns\n"
          "q_out (None without q).");
    m.def("kv4_read", &kv4_read, py::arg("pages"), py::arg("block_table"), py::arg("cu_seqlens"), py::arg("kv_len"),
          py::arg("rows"), py::arg("head_dim"), py::arg("dtype"), py::arg("k_out") = none, py::arg("v_out") = none,
          py::arg("stream") = none,
          "The values (k, v), each [rows, kv_heads, head_dim] of dtype, of the last\n"
          "cu_seqlens[b + 1] - cu_seqlens[b] slots of every sequence; rows = cu_seqlens[batch].");
    m.def("kv4_attention", &kv4_attention, py::arg("q"), py::arg("pages"), py::arg("block_table"),
          py::arg("cu_seqlens"), py::arg("kv_len"), py::arg("max_q"), py::arg("max_kv"), py::arg("scale") = none,
          py::arg("causal") = true, py::arg("window") = 0, py::arg("out") = none, py::arg("return_lse") = false,
          py::arg("lse") = none, py::arg("workspace") = none, py::arg("stream") = none,
          "softmax(scale q . k) v over the cache for q [T, q_heads, D] (scale: 1 / sqrt(D) unless given).  A token\n"
          "sees the slots up to its own (with causal=False all of its sequence's; with a window only that many\n"
          "last ones); one that sees none gets zeros.  max_q, max_kv: at least the most new tokens and slots of\n"
          "any sequence.  Returns out, or (out, lse) with return_lse (lse fp32 [T, q_heads], -inf where nothing\n"
          "is seen).");
    m.def("kv4_tree_attention", &kv4_tree_attention, py::arg("q"), py::arg("pages"), py::arg("block_table"),
          py::arg("cu_seqlens"), py::arg("kv_len"), py::arg("tree"), py::arg("max_q"), py::arg("max_kv"),
          py::arg("scale") = none, py::arg("window") = 0, py::arg("out") = none, py::arg("return_lse") = false,
          py::arg("lse") = none, py::arg("workspace") = none, py::arg("stream") = none,
          "kv4_attention for new tokens that are a tree of drafts, up to 64 a sequence: bit j of a token's word in\n"
          "tree (int64 [T]) says that it descends from its sequence's new token j, an earlier one.  A token sees the\n"
          "slots before the new ones, those of the tokens that it descends from, and its own.  window: 0, or at\n"
          "least 64, counted along a token's path.");
    m.def("kv4_attention_mass", &kv4_attention_mass, py::arg("q"), py::arg("pages"), py::arg("block_table"),
          py::arg("cu_seqlens"), py::arg("kv_len"), py::arg("lse"), py::arg("acc"), py::arg("max_q"),
          py::arg("max_kv"), py::arg("scale") = none, py::arg("causal") = true, py::arg("window") = 0,
          py::arg("stream") = none,
          "Add to acc (fp32 [batch, kv_heads, slots], slots >= max_kv) the attention weight that every cached slot\n"
          "got from this call's queries: the sum of exp(scale q . k - lse) over the tokens that see it and the\n"
          "query heads of its head.  The other arguments as kv4_attention had and gave them.  Returns acc.");
    m.def("kv4_evict", &kv4_evict, py::arg("pages"), py::arg("block_table"), py::arg("kv_len"), py::arg("acc"),
          py::arg("budget"), py::arg("recent"), py::arg("dst_table"), py::arg("head_dim"), py::arg("max_kv"),
          py::arg("stream") = none,
          "Cut every sequence and head to at most budget slots: the last `recent` and, of the others, those with\n"
          "the largest acc (fp32 [batch, kv_heads, slots >= max_kv]; equal ones: the lowest slots).  What is kept\n"
          "is copied, in its order, into the pages of dst_table (int32 [batch, pages]; in the same tensor, none of\n"
          "them in use by block_table).  Returns (kept int32 [batch, kv_heads, budget], new_len int32 [batch], acc\n"
          "of the kept slots fp32 [batch, kv_heads, budget]); -1 and 0 beyond new_len.");
}
