// common.hpp -- what the Python bindings share: checks of tensors, the stream and
// device of a call, workspaces. Each binding's module holds its own copy.
#pragma once

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "../../include/bqm.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

// Given by the package when it loads this module.
PyObject *g_error, *g_raw_stream;

[[maybe_unused]] void set_common(py::object error, py::object raw_stream)
{
    g_error = error.release().ptr();
    g_raw_stream = raw_stream.release().ptr();
}

std::string text(const char *name, const std::string &rest) { return std::string(name) + rest; }

[[noreturn]] void bad_value(const std::string &s) { throw py::value_error(s); }
[[noreturn]] void bad_type(const std::string &s) { throw py::type_error(s); }

void done(const char *fn, int status)
{
    if (status == BQM_OK)
        return;
    py::object e = py::reinterpret_borrow<py::object>(g_error)(fn, status);
    PyErr_SetObject(g_error, e.ptr());
    throw py::error_already_set();
}

int code_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat:
        return BQM_DTYPE_F32;
    case at::kHalf:
        return BQM_DTYPE_F16;
    case at::kBFloat16:
        return BQM_DTYPE_BF16;
    default:
        bad_type(std::string("dtype ") + at::toString(t) +
                 ": float32, float16 or bfloat16 expected");
    }
}

// Checks a tensor; dev < 0: any GPU; dims < 0: any number.
void gpu(const Tensor &t, const char *name, int64_t dims, int dev = -1)
{
    if (!t.defined() || !t.is_cuda())
        bad_type(text(name, " must be a GPU tensor"));
    if (dims >= 0 && t.dim() != dims)
        bad_value(text(name, " has " + std::to_string(t.dim()) + " dimensions, expected " +
                                 std::to_string(dims)));
    if (dev >= 0 && t.get_device() != dev)
        bad_value(text(name, " is on GPU " + std::to_string(t.get_device()) + ", expected " +
                                 std::to_string(dev)));
}

void typed(const Tensor &t, const char *name, at::ScalarType type)
{
    if (t.scalar_type() != type)
        bad_type(text(name, std::string(" has dtype ") + at::toString(t.scalar_type()) +
                                ", expected " + at::toString(type)));
}

// A contiguous int32 vector of n entries.
int32_t *ints(const Tensor &t, const char *name, int64_t n, int dev)
{
    gpu(t, name, 1, dev);
    typed(t, name, at::kInt);
    if (t.size(0) != n || (n > 1 && t.stride(0) != 1))
        bad_value(text(name, " must be a contiguous vector of " + std::to_string(n)));
    return static_cast<int32_t *>(t.data_ptr());
}

std::optional<at::ScalarType> dtype_of(const py::object &d)
{
    if (d.is_none())
        return std::nullopt;
    if (!THPDtype_Check(d.ptr()))
        bad_type("a torch.dtype is expected");
    return reinterpret_cast<THPDtype *>(d.ptr())->scalar_type;
}

// Where a call runs: on the GPU of its tensors, on the stream given or on the GPU's
// current one. Both are the current ones while this lives, so that what the call
// allocates is the stream's own: memory of another stream may be in use there still,
// by kernels of a call that has returned.
struct On {
    c10::OptionalDeviceGuard device;
    c10::OptionalStreamGuard guard;
    std::optional<c10::Stream> caller;  // the stream that was current, where that is another
    void *p;

    On(const py::object &stream, int dev)
    {
        if (stream.is_none()) {
            device.reset_device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
        } else {
            const auto s = c10::Stream::unpack3(
                stream.attr("stream_id").cast<int64_t>(),
                (c10::DeviceIndex)stream.attr("device_index").cast<int>(),
                (c10::DeviceType)stream.attr("device_type").cast<int>());
            if (s.device_type() != c10::kCUDA || s.device_index() != dev)
                bad_value("stream is not one of GPU " + std::to_string(dev));
            guard.reset_stream(s);
            if (*guard.original_stream() != s)
                caller = guard.original_stream();
        }
        const py::object raw =
            stream.is_none()
                ? py::reinterpret_steal<py::object>(PyObject_CallFunction(g_raw_stream, "i", dev))
                : stream.attr("cuda_stream");
        if (!raw)
            throw py::error_already_set();
        p = PyLong_AsVoidPtr(raw.ptr());
        if (PyErr_Occurred())
            throw py::error_already_set();
    }

    // A new output: the caller's current stream will use it too, and the allocator is
    // told so.
    Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Tensor &like) const
    {
        Tensor t = at::empty(sizes, like.options().dtype(type));
        if (caller)
            t.record_stream(*caller);
        return t;
    }
};

// A workspace: the caller's, or one of this call alone, which the stream's next call
// may have again.
struct Scratch {
    Tensor t;
    void *p = nullptr;
    size_t bytes = 0;

    // (`On` stands for its own lifetime: the memory is taken from its stream's)
    Scratch(const OptTensor &given, size_t need, const Tensor &like, const On &)
    {
        if (given) {
            t = *given;
            gpu(t, "workspace", 1, like.get_device());
            typed(t, "workspace", at::kByte);
            if ((size_t)t.size(0) < need || (t.size(0) > 1 && t.stride(0) != 1))
                bad_value("workspace must be " + std::to_string(need) + " contiguous bytes");
        } else if (need == 0) {
            return;
        } else {
            t = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
        }
        p = t.data_ptr();
        bytes = (size_t)t.size(0);
    }
};

}  // namespace
