// What the Python bindings of the operators share: argument checks, the stream of a call, errors.
#pragma once

#include <torch/extension.h>

#include <ATen/hip/impl/HIPGuardImplMasqueradingAsCUDA.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>

#include <cmath>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/w4a16.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;
using StreamGuard = c10::hip::HIPStreamGuardMasqueradingAsCUDA;

namespace binding {

[[noreturn]] inline void refuse(const std::string &what) { throw py::value_error(what); }

inline void check(int status, const char *what) {
    if (status == W4A16_OK) return;
    const py::object type = py::module_::import("int4_weight_only_w4a16_amd").attr("W4A16Error");
    const py::object error = type(status, what);
    PyErr_SetObject(type.ptr(), error.ptr());
    throw py::error_already_set();
}

inline unsigned type_flag(at::ScalarType t, const char *of = "q, k and v") {
    if (t == at::kBFloat16) return W4A16_X_BF16;
    if (t != at::kHalf) refuse(std::string(of) + " must be float16 or bfloat16");
    return 0;
}

// The stream a call runs on, and while this lives the device and, for a stream that the caller
// named, the stream that new tensors belong to.
class On {
  public:
    On(const Tensor &t, const py::object &stream) : device_(t.device()) {
        if (stream.is_none()) {
            handle_ = c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream();
            return;
        }
        const py::object raw = py::isinstance<py::int_>(stream) ? stream : stream.attr("cuda_stream");
        handle_ = reinterpret_cast<hipStream_t>(raw.cast<uintptr_t>());
        guard_.emplace(c10::hip::getStreamFromExternalMasqueradingAsCUDA(handle_, t.device().index()));
    }
    void *stream() const { return handle_; }

  private:
    c10::OptionalDeviceGuard device_;
    hipStream_t handle_;
    std::optional<StreamGuard> guard_;
};

// Token stride of a [tokens, heads, channels] tensor whose heads and channels are contiguous.
inline int64_t heads_stride(const char *name, const Tensor &t, const Tensor *like = nullptr) {
    if (t.dim() != 3 || !t.is_cuda() || t.stride(2) != 1 || t.stride(1) != t.size(2))
        refuse(std::string(name) + " must be a device tensor [tokens, heads, channels], contiguous but for the "
               "stride between tokens");
    if (like && (t.scalar_type() != like->scalar_type() || t.device() != like->device()))
        refuse(std::string(name) + " must have the type and device of the other inputs");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);     // (a single token may carry any stride)
}

inline void *plain(const char *name, const Tensor &t, at::ScalarType type, const at::Device &device,
            std::initializer_list<int64_t> shape = {}) {
    if (t.scalar_type() != type || t.device() != device || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor on " + device.str());
    if (shape.size() && t.sizes() != at::IntArrayRef(shape)) refuse(std::string(name) + " has the wrong shape");
    return t.data_ptr();
}

}  // namespace binding
