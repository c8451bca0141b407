// Python binding of the short convolution and the gated delta rule, in the module of the
// cache's operators.

#include "binding.hpp"

namespace {

using namespace binding;

// The sequences of a call and its pool of states.
struct Sequences {
    int64_t batch;
    const int32_t *index, *seen, *cu;
    const int64_t *tree;
};

Sequences sequences_of(const Tensor &like, int64_t T, const Tensor &state_index, const Tensor &cu_seqlens,
                       const MaybeTensor &seen, const MaybeTensor &tree) {
    if (state_index.dim() != 1) refuse("state_index must be [batch]");
    Sequences s{state_index.size(0), nullptr, nullptr, nullptr, nullptr};
    s.index = static_cast<int32_t *>(plain("state_index", state_index, at::kInt, like.device()));
    s.cu = static_cast<int32_t *>(plain("cu_seqlens", cu_seqlens, at::kInt, like.device(), {s.batch + 1}));
    if (seen) s.seen = static_cast<int32_t *>(plain("seen", *seen, at::kInt, like.device(), {s.batch}));
    if (tree) s.tree = static_cast<int64_t *>(plain("tree", *tree, at::kLong, like.device(), {T}));
    return s;
}

// Row stride of a [rows, columns] tensor whose columns are contiguous.
int64_t rows_stride(const char *name, const Tensor &t, int64_t rows, int64_t columns, at::ScalarType type,
                    const at::Device &device) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != columns || t.scalar_type() != type ||
        t.device() != device || !t.is_cuda() || (columns > 1 && t.stride(1) != 1))
        refuse(std::string(name) + " must be a " + c10::toString(type) + " device tensor [" + std::to_string(rows) +
               ", " + std::to_string(columns) + "], contiguous but for the stride between rows");
    return rows > 1 ? t.stride(0) : columns;     // (a single row may carry any stride)
}

Tensor short_conv(const Tensor &x, const Tensor &weight, const Tensor &state, const Tensor &state_index,
                  const Tensor &cu_seqlens, int64_t max_q, const MaybeTensor &bias, const MaybeTensor &seen,
                  const MaybeTensor &tree, bool silu, const MaybeTensor &out, const py::object &stream) {
    if (x.dim() != 2 || weight.dim() != 2 || state.dim() != 3)
        refuse("x must be [tokens, channels], weight [channels, width] and state [states, width - 1, channels]");
    const int64_t T = x.size(0), C = x.size(1), W = weight.size(1);
    const unsigned flags = type_flag(x.scalar_type(), "x") | (silu ? W4A16_SILU : 0);
    const int64_t xs = rows_stride("x", x, T, C, x.scalar_type(), x.device());
    const auto *w = static_cast<float *>(plain("weight", weight, at::kFloat, x.device(), {C, W}));
    const float *bias_ptr = nullptr;
    if (bias) bias_ptr = static_cast<float *>(plain("bias", *bias, at::kFloat, x.device(), {C}));
    void *states = plain("state", state, x.scalar_type(), x.device(), {state.size(0), W - 1, C});
    const Sequences s = sequences_of(x, T, state_index, cu_seqlens, seen, tree);
    const On on(x, stream);
    const Tensor y = out ? *out : at::empty({T, C}, x.options());
    check(w4a16_short_conv(x.data_ptr(), xs, w, bias_ptr, states, s.index, s.seen, s.cu, s.tree, y.data_ptr(),
                           rows_stride("out", y, T, C, x.scalar_type(), x.device()), T, C, W, state.size(0), s.batch,
                           max_q, flags, on.stream()),
          "w4a16_short_conv");
    return y;
}

Tensor gated_delta_rule(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &a, const Tensor &b,
                        const Tensor &state, const Tensor &state_index, const Tensor &cu_seqlens, int64_t max_q,
                        const MaybeTensor &a_log, const MaybeTensor &dt_bias, const MaybeTensor &seen,
                        const MaybeTensor &tree, std::optional<double> scale, bool unit_qk, double eps,
                        const MaybeTensor &out, const MaybeTensor &workspace, const py::object &stream) {
    const int64_t qs = heads_stride("q", q), ks = heads_stride("k", k, &q), vs = heads_stride("v", v, &q);
    const int64_t T = q.size(0), hk = q.size(1), dk = q.size(2), hv = v.size(1), dv = v.size(2);
    if (k.sizes() != q.sizes() || v.size(0) != T)
        refuse("q and k must be [tokens, key heads, channels], v [tokens, value heads, channels] of the same tokens");
    const unsigned flags = type_flag(q.scalar_type()) | (unit_qk ? W4A16_UNIT_QK : 0);
    if (a_log.has_value() != dt_bias.has_value()) refuse("a_log and dt_bias go together");
    const at::ScalarType gates = a_log ? q.scalar_type() : at::kFloat;
    const int64_t as = rows_stride("a", a, T, hv, gates, q.device()), bs = rows_stride("b", b, T, hv, gates, q.device());
    const float *log_ptr = nullptr, *bias_ptr = nullptr;
    if (a_log) {
        log_ptr = static_cast<float *>(plain("a_log", *a_log, at::kFloat, q.device(), {hv}));
        bias_ptr = static_cast<float *>(plain("dt_bias", *dt_bias, at::kFloat, q.device(), {hv}));
    }
    if (state.dim() != 4) refuse("state must be [states, value heads, key channels, value channels]");
    auto *states = static_cast<float *>(plain("state", state, at::kFloat, q.device(), {state.size(0), hv, dk, dv}));
    const Sequences s = sequences_of(q, T, state_index, cu_seqlens, seen, tree);
    const On on(q, stream);
    const Tensor o = out ? *out : at::empty({T, hv, dv}, q.options());
    if (o.dim() != 3 || o.size(0) != T || o.size(1) != hv || o.size(2) != dv)
        refuse("out must be [tokens, value heads, channels]");
    const size_t need = w4a16_delta_rule_workspace_bytes(s.batch, T, hk, hv, dk, dv, max_q, s.tree != nullptr);
    Tensor ws;
    if (workspace) {
        ws = *workspace;
        plain("workspace", ws, ws.scalar_type(), q.device());     // (any type: bytes are what counts)
    } else if (need) {
        ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    }
    check(w4a16_delta_rule(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, a.data_ptr(), as, b.data_ptr(), bs,
                           log_ptr, bias_ptr, states, s.index, s.seen, s.cu, s.tree, o.data_ptr(),
                           heads_stride("out", o, &q), T, hk, hv, dk, dv, state.size(0), s.batch, max_q,
                           (float)(scale ? *scale : 1.0 / std::sqrt((double)dk)), (float)eps, flags,
                           ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, on.stream()),
          "w4a16_delta_rule");
    return o;
}

}  // namespace

void bind_delta(py::module_ &m) {
    const auto none = py::none();
    m.def("short_conv", &short_conv, py::arg("x"), py::arg("weight"), py::arg("state"), py::arg("state_index"),
          py::arg("cu_seqlens"), py::arg("max_q"), py::arg("bias") = none, py::arg("seen") = none,
          py::arg("tree") = none, py::arg("silu") = true, py::arg("out") = none, py::arg("stream") = none,
          "Causal convolution of each channel over the last `width` rows (weight fp32 [channels, width], the last\n"
          "column the token's own; width 2 to 4) of x [T, channels], with SiLU unless silu=False.  Sequence b is\n"
          "rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1; the rows before its first are state[state_index[b]]\n"
          "([states, width - 1, channels], x's type), or zeros where seen[b] (int32 [batch], None: all have) is 0,\n"
          "and that state becomes the sequence's last width - 1 rows.  max_q: at least the most tokens of any\n"
          "sequence.  tree (int64 [T]): the tokens are a tree of drafts as in kv4_tree_attention, the rows before\n"
          "one those that it descends from, and the state stays as it is.  Returns out [T, channels].");
    m.def("gated_delta_rule", &gated_delta_rule, py::arg("q"), py::arg("k"), py::arg("v"), py::arg("a"), py::arg("b"),
          py::arg("state"), py::arg("state_index"), py::arg("cu_seqlens"), py::arg("max_q"), py::arg("a_log") = none,
          py::arg("dt_bias") = none, py::arg("seen") = none, py::arg("tree") = none, py::arg("scale") = none,
          py::arg("unit_qk") = false, py::arg("eps") = 1e-6, py::arg("out") = none, py::arg("workspace") = none,
          py::arg("stream") = none,
          "For each token, S <- e^g S, u = beta (v - S^T k), S <- S + k u^T, out = scale S^T q, with S the state\n"
          "(fp32 [states, value heads, key channels, value channels]) that state_index (int32 [batch]) names for the\n"
          "sequence, zeros where seen (int32 [batch], None: nowhere) is 0; it is left as the last token leaves it.\n"
          "q, k [T, key heads, 64 or 128], v [T, value heads, 64, 128, 192 or 256]; value head h uses key head\n"
          "h // (value heads / key heads); with unit_qk q and k are brought to unit length, x / sqrt(sum x^2 + eps).\n"
          "Gates: with a_log and dt_bias (fp32 [value heads]) g = -exp(a_log) softplus(a + dt_bias) and\n"
          "beta = sigmoid(b), a and b [T, value heads] of q's type; without, a is g (not positive) and b beta, fp32.\n"
          "scale: 1 / sqrt(key channels) unless given.  max_q: at least the most tokens of any sequence.  tree\n"
          "(int64 [T]): the tokens are a tree of drafts as in kv4_tree_attention, each continues the state that the\n"
          "last token it descends from left, and the states stay as they are.  One long sequence beside many of a few\n"
          "tokens is better two calls.  Returns out [T, value heads, value channels].");
}
