// tokens.cpp -- Python binding of the token side of include/bqm.h: checks arguments,
// allocates outputs and calls the C ABI. Native for the same reason as the attention
// side's: single tokens' kernels take a few us.
#include "common.hpp"

namespace {

// A contiguous tensor of the size given.
void whole(const Tensor &t, const char *name, at::IntArrayRef sizes, int dev)
{
    gpu(t, name, (int64_t)sizes.size(), dev);
    if (t.sizes() != sizes || !t.is_contiguous()) {
        std::string s;
        for (const int64_t n : sizes)
            s += (s.empty() ? "" : ", ") + std::to_string(n);
        bad_value(text(name, " must be contiguous [" + s + "]"));
    }
}

// A contiguous vector of n entries, or nothing.
template <class T>
T *vector(const OptTensor &t, const char *name, at::ScalarType type, int64_t n, int dev)
{
    if (!t)
        return nullptr;
    gpu(*t, name, 1, dev);
    typed(*t, name, type);
    if (t->size(0) != n || (n > 1 && t->stride(0) != 1))
        bad_value(text(name, " must be a contiguous vector of " + std::to_string(n)));
    return static_cast<T *>(t->data_ptr());
}

// rms_norm's arguments but its outputs, and where the sums go.
struct Norm {
    int64_t T, K;
    int dev;
    On on;
    Tensor stream;  // what the sums are afterwards: x itself where nothing is added
    const void *add = nullptr;
    void *sum = nullptr;
    float *gain;
    int dtype, add_dtype = 0;

    static int check(const Tensor &x)
    {
        gpu(x, "x", 2);
        if (!x.is_contiguous())
            bad_value("x must be contiguous");
        return x.get_device();
    }

    Norm(const Tensor &x, const OptTensor &gain_, const OptTensor &add_, const OptTensor &sum_out,
         const py::object &stream_)
        : T(0), K(0), dev(check(x)), on(stream_, dev), stream(x)
    {
        T = x.size(0);
        K = x.size(1);
        dtype = code_of(x.scalar_type());
        gain = vector<float>(gain_, "gain", at::kFloat, K, dev);
        if (add_) {
            whole(*add_, "add", x.sizes(), dev);
            add_dtype = code_of(add_->scalar_type());
            add = add_->data_ptr();
        }
        if (sum_out) {
            whole(*sum_out, "sum_out", x.sizes(), dev);
            typed(*sum_out, "sum_out", x.scalar_type());
            stream = *sum_out;
        } else if (add_) {
            stream = on.empty(x.sizes(), x.scalar_type(), x);
        }
        if (sum_out || add_)
            sum = stream.data_ptr();
    }

    void run(const Tensor &x, void *y, int y_dtype, void *a, double eps) const
    {
        if (T)
            done("rms_norm", rms_norm(x.data_ptr(), add, gain, sum, y, a, T, K, eps, dtype,
                                      add_dtype, y_dtype, on.p));
    }
};

py::tuple rms_norm_(const Tensor &x, const OptTensor &gain, const OptTensor &add, double eps,
                    const OptTensor &sum_out, const OptTensor &out_, const py::object &out_dtype,
                    const py::object &stream)
{
    const auto want = dtype_of(out_dtype);
    const Norm n(x, gain, add, sum_out, stream);
    const Tensor out = out_ ? *out_ : n.on.empty(x.sizes(), want.value_or(x.scalar_type()), x);
    if (out_) {
        whole(out, "out", x.sizes(), n.dev);
        if (want)
            typed(out, "out", *want);
    }
    n.run(x, out.data_ptr(), code_of(out.scalar_type()), nullptr, eps);
    return py::make_tuple(out, n.stream);
}

py::tuple rms_norm_q8_1_(const Tensor &x, const OptTensor &gain, const OptTensor &add, double eps,
                         const OptTensor &sum_out, const OptTensor &out_, const py::object &stream)
{
    const Norm n(x, gain, add, sum_out, stream);
    const Tensor out = out_ ? *out_ : n.on.empty({n.T, n.K / 32 * 36}, at::kByte, x);
    if (out_) {
        whole(out, "out", {n.T, n.K / 32 * 36}, n.dev);
        typed(out, "out", at::kByte);
    }
    n.run(x, nullptr, 0, out.data_ptr(), eps);
    return py::make_tuple(out, n.stream);
}

struct Q4Matrix {
    Tensor codes, scales;
    OptTensor zeros;
    bqm_q4_matrix m;
    int dev;

    Q4Matrix(const Tensor &c, const Tensor &s, const OptTensor &z) : codes(c), scales(s), zeros(z)
    {
        gpu(codes, "codes", 2);
        typed(codes, "codes", at::kByte);
        dev = codes.get_device();
        gpu(scales, "scales", 2, dev);
        typed(scales, "scales", at::kHalf);
        if (!codes.is_contiguous() || !scales.is_contiguous())
            bad_value("codes and scales must be contiguous");
        const int64_t N = codes.size(0), K = 2 * codes.size(1), groups = scales.size(1);
        if (scales.size(0) != N || groups < 1 || K % groups != 0 || K / groups > 128)
            bad_value("scales must be [rows, values of a row / 32, 64 or 128]");
        if (zeros) {
            whole(*zeros, "zeros", scales.sizes(), dev);
            typed(*zeros, "zeros", at::kChar);
        }
        m = {codes.data_ptr(), scales.data_ptr(),
             zeros ? static_cast<int8_t *>(zeros->data_ptr()) : nullptr, N, K,
             (int32_t)(K / groups)};
    }
};

Q4Matrix q4_quantize_(const Tensor &x, int64_t group, bool zeros, const py::object &stream)
{
    gpu(x, "x", 2);
    if (!x.is_contiguous())
        bad_value("x must be contiguous");
    const int64_t N = x.size(0), K = x.size(1);
    if ((group != 32 && group != 64 && group != 128) || K < 1 || K % group != 0)
        bad_value("x must have rows of whole groups of 32, 64 or 128");
    const On on(stream, x.get_device());
    const int dtype = code_of(x.scalar_type());
    OptTensor z;
    if (zeros)
        z = on.empty({N, K / group}, at::kChar, x);
    Q4Matrix m(on.empty({N, K / 2}, at::kByte, x), on.empty({N, K / group}, at::kHalf, x), z);
    done("q4_quantize", q4_quantize(x.data_ptr(), &m.m, dtype, on.p));
    return m;
}

Tensor mm_q4_(const Q4Matrix &m, const Tensor &a, const OptTensor &out_,
              const OptTensor &workspace, const py::object &stream)
{
    gpu(a, "a", 2, m.dev);
    typed(a, "a", at::kByte);
    const int64_t T = a.size(0);
    whole(a, "a", {T, m.m.K / 32 * 36}, m.dev);
    const On on(stream, m.dev);
    const Tensor out = out_ ? *out_ : on.empty({T, m.m.N}, at::kFloat, a);
    if (out_) {
        whole(out, "out", {T, m.m.N}, m.dev);
        typed(out, "out", at::kFloat);
    }
    if (T) {
        const Scratch w(workspace, mm_q4_workspace_bytes(&m.m, T), a, on);
        done("mm_q4", mm_q4(&m.m, a.data_ptr(), static_cast<float *>(out.data_ptr()), T, w.p,
                            w.bytes, on.p));
    }
    return out;
}

Tensor q4_dequantize_(const Q4Matrix &m, const OptTensor &rows, double scale,
                      const py::object &dtype, const OptTensor &out_, const py::object &stream)
{
    const int64_t n = rows ? rows->dim() == 1 ? rows->size(0) : -1 : m.m.N;
    const int32_t *ids = vector<int32_t>(rows, "rows", at::kInt, n, m.dev);
    const auto want = dtype_of(dtype);
    const On on(stream, m.dev);
    const Tensor out =
        out_ ? *out_ : on.empty({n, m.m.K}, want.value_or(at::kHalf), m.codes);
    if (out_) {
        whole(out, "out", {n, m.m.K}, m.dev);
        if (want)
            typed(out, "out", *want);
    }
    const int to = code_of(out.scalar_type());
    if (n)
        done("q4_dequantize",
             q4_dequantize(&m.m, ids, out.data_ptr(), n, (float)scale, to, on.p));
    return out;
}

py::tuple sample_(const Tensor &logits, const Tensor &u, const OptTensor &temperature,
                  const OptTensor &top_k, const OptTensor &top_p, const OptTensor &min_p,
                  const OptTensor &out_, const OptTensor &logprobs_, const OptTensor &workspace,
                  const py::object &stream)
{
    gpu(logits, "logits", 2);
    const int dev = logits.get_device();
    const int64_t T = logits.size(0), V = logits.size(1);
    if (V > 1 && logits.stride(1) != 1)
        bad_value("a row of logits must be contiguous");
    const int dtype = code_of(logits.scalar_type());
    const float *heat = vector<float>(temperature, "temperature", at::kFloat, T, dev);
    const int32_t *k = vector<int32_t>(top_k, "top_k", at::kInt, T, dev);
    const float *p = vector<float>(top_p, "top_p", at::kFloat, T, dev);
    const float *least = vector<float>(min_p, "min_p", at::kFloat, T, dev);
    const float *random = vector<float>(u, "u", at::kFloat, T, dev);
    const On on(stream, dev);
    const Tensor out = out_ ? *out_ : on.empty({T}, at::kInt, logits);
    const Tensor logprobs = logprobs_ ? *logprobs_ : on.empty({T}, at::kFloat, logits);
    int32_t *tokens = ints(out, "out", T, dev);
    float *lp = vector<float>(logprobs, "logprobs", at::kFloat, T, dev);
    if (T) {
        const Scratch w(workspace, sample_workspace_bytes(T, V), logits, on);
        done("sample", sample(logits.data_ptr(), logits.stride(0), heat, k, p, least, random,
                              tokens, lp, T, V, dtype, w.p, w.bytes, on.p));
    }
    return py::make_tuple(out, logprobs);
}

}  // namespace

PYBIND11_MODULE(_tokens, m)
{
    const py::arg_v stream("stream", py::none()), out("out", py::none());
    const py::arg_v gain("gain", py::none()), add("add", py::none()), sum("sum_out", py::none());
    m.def("set_python", &set_common);
    m.def("rms_norm", &rms_norm_, py::arg("x"), gain, add, py::arg("eps") = 1e-6, sum, out,
          py::arg("out_dtype") = py::none(), stream,
          "(y, s): s = x + add in x's type (x itself where nothing is added), y = s / sqrt(mean of s^2 + "
          "eps) * gain.\nx [T, K], add of the same shape, gain fp32 [K], all contiguous; y in x's type or "
          "out_dtype. sum_out takes s\n(x itself: in place).");
    m.def("rms_norm_q8_1", &rms_norm_q8_1_, py::arg("x"), gain, add, py::arg("eps") = 1e-6, sum, out,
          stream,
          "(a, s) as rms_norm, y as Q8_1 blocks: uint8 [T, K / 32 * 36], the products' activations. A NaN of "
          "y is 0 in\nthem, as in q8_1_quantize.");
    py::class_<Q4Matrix>(m, "Q4Matrix",
                         "A matrix in 4 bits: codes uint8 [rows, values / 2] (each run of 16 bytes 32 "
                         "values: low halves the first 16,\nhigh halves the rest, two's complement), scales "
                         "float16 [rows, groups] and, or None, zeros int8 [rows, groups];\nvalue = scale * "
                         "(code - zero), groups of 32, 64 or 128.")
        .def(py::init<const Tensor &, const Tensor &, const OptTensor &>(), py::arg("codes"),
             py::arg("scales"), py::arg("zeros") = py::none())
        .def_readonly("codes", &Q4Matrix::codes)
        .def_readonly("scales", &Q4Matrix::scales)
        .def_readonly("zeros", &Q4Matrix::zeros)
        .def_property_readonly("N", [](const Q4Matrix &q) { return q.m.N; })
        .def_property_readonly("K", [](const Q4Matrix &q) { return q.m.K; })
        .def_property_readonly("group", [](const Q4Matrix &q) { return q.m.group; });
    m.def("q4_quantize", &q4_quantize_, py::arg("x"), py::arg("group") = 64,
          py::arg("zeros") = false, stream,
          "The Q4Matrix nearest to x [N, K] (float32, float16 or bfloat16), with zeros for groups that are "
          "not centred.");
    m.def("mm_q4_workspace_bytes",
          [](const Q4Matrix &q, int64_t T) { return mm_q4_workspace_bytes(&q.m, T); }, py::arg("m"),
          py::arg("T"),
          "Bytes of the uint8 tensor that mm_q4(..., workspace=) takes for up to T columns (0: none).");
    m.def("mm_q4", &mm_q4_, py::arg("m"), py::arg("a"), out, py::arg("workspace") = py::none(),
          stream,
          "y fp32 [T, N] = a Q4Matrix times T Q8_1 activation columns a, uint8 [T, K / 32 * 36].");
    m.def("q4_dequantize", &q4_dequantize_, py::arg("m"), py::arg("rows") = py::none(),
          py::arg("scale") = 1.0, py::arg("dtype") = py::none(), out, stream,
          "Rows rows int32 [n] (or all) of a Q4Matrix, times scale: [n, K] of dtype (float16 by default). A "
          "table's look-up.");
    m.def("sample", &sample_, py::arg("logits"), py::arg("u"), py::arg("temperature") = py::none(),
          py::arg("top_k") = py::none(), py::arg("top_p") = py::none(),
          py::arg("min_p") = py::none(), out, py::arg("logprobs") = py::none(),
          py::arg("workspace") = py::none(), stream,
          "(tokens int32 [T], logprobs fp32 [T]): the next token of each row of logits [T, V], for random "
          "numbers u\nfp32 [T] of [0, 1). temperature (0: the largest), top_p, min_p fp32 [T] and top_k int32 "
          "[T] as in include/bqm.h;\n-1 for a row of -inf.");
}
