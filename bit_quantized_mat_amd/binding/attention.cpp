// attention.cpp -- Python binding of the attention side of include/bqm.h:
// checks arguments, allocates outputs and calls the C ABI.
//
// Native, because the smallest of these kernels take 2 to 8 us: the same checks
// in Python over ctypes took 12 to 14 us a call.
#include <cmath>

#include "common.hpp"

namespace {

PyObject *g_pages;

void set_python(py::object error, py::object pages, py::object raw_stream)
{
    set_common(std::move(error), std::move(raw_stream));
    g_pages = pages.release().ptr();
}

// [tokens, heads, values] with contiguous values.
void heads(const Tensor &t, const char *name, int dev = -1)
{
    gpu(t, name, 3, dev);
    if (t.size(2) > 1 && t.stride(2) != 1)
        bad_value(text("the values of a head of ", std::string(name) + " must be contiguous"));
}

int32_t to_int32(int64_t n, const char *name)
{
    if (n < INT32_MIN || n > INT32_MAX)
        bad_value(text(name, " is out of range"));
    return (int32_t)n;
}

struct KvCache {
    Tensor k, v;
    bqm_kv_cache c;
    int dev;

    KvCache(const Tensor &k_, const Tensor &v_) : k(k_), v(v_)
    {
        gpu(k, "k", -1);
        dev = k.get_device();
        gpu(v, "v", k.dim(), dev);
        typed(v, "v", k.scalar_type());
        if (k.scalar_type() != at::kHalf && k.scalar_type() != at::kBFloat16)
            bad_type(std::string("k has dtype ") + at::toString(k.scalar_type()) +
                     ", expected float16 or bfloat16");
        const int64_t n = k.dim();
        if (n != 4 && n != 5)
            bad_value("k has " + std::to_string(n) + " dimensions, expected 4 or 5");
        if (k.sizes() != v.sizes() || k.strides() != v.strides())
            bad_value("k and v differ in shape or strides");
        if (k.size(n - 1) > 1 && k.stride(n - 1) != 1)
            bad_value("the values of a head must be contiguous");
        if (k.size(n - 3) > INT32_MAX || k.size(n - 2) > INT32_MAX || k.size(n - 1) > INT32_MAX)
            bad_value("k is too large");
        c = {k.data_ptr(), v.data_ptr(), n == 5 ? k.stride(0) : 0, k.stride(n - 4),
             k.stride(n - 3), k.stride(n - 2), n == 5 ? k.size(0) : 1, k.size(n - 4),
             (int32_t)k.size(n - 3), (int32_t)k.size(n - 2), (int32_t)k.size(n - 1),
             code_of(k.scalar_type())};
    }

    KvCache layer(int64_t i) const { return k.dim() == 5 ? KvCache(k.select(0, i), v.select(0, i)) : *this; }
};

struct KvBatch {
    Tensor table, kv_lens, q_starts;
    std::optional<int64_t> max_q, max_kv;
    bqm_kv_batch b;
    int dev;

    KvBatch(const Tensor &t, const Tensor &l, const Tensor &s, std::optional<int64_t> mq,
            std::optional<int64_t> mkv)
        : table(t), kv_lens(l), q_starts(s), max_q(mq), max_kv(mkv)
    {
        gpu(table, "table", 2);
        typed(table, "table", at::kInt);
        dev = table.get_device();
        if (table.size(1) > 1 && table.stride(1) != 1)
            bad_value("the table's rows must be contiguous");
        const int64_t n = table.size(0);
        b = {static_cast<int32_t *>(table.data_ptr()), ints(kv_lens, "kv_lens", n, dev),
             ints(q_starts, "q_starts", n + 1, dev), table.stride(0), 0,
             to_int32(n, "the table"), to_int32(table.size(1), "the table"), 0, 0};
    }

    bqm_kv_batch of(int64_t total_q, const KvCache &cache) const
    {
        if (dev != cache.dev)
            bad_value("the batch is on GPU " + std::to_string(dev) + ", expected " +
                      std::to_string(cache.dev));
        bqm_kv_batch r = b;
        r.total_q = total_q;
        r.max_q = to_int32(max_q.value_or(total_q), "max_q");
        r.max_kv = to_int32(max_kv.value_or(std::min<int64_t>(
                                (int64_t)b.max_pages * cache.c.page_size, 1ll << 30)),
                            "max_kv");
        return r;
    }
};

struct Angles {
    float *p;
    int64_t n_pos, n_freq;

    Angles(const Tensor &t, int dev)
    {
        gpu(t, "table", 3, dev);
        typed(t, "table", at::kFloat);
        if (t.size(2) != 2 || !t.is_contiguous())
            bad_value("table must be contiguous [n_pos, n_freq, 2]");
        p = static_cast<float *>(t.data_ptr());
        n_pos = t.size(0);
        n_freq = t.size(1);
    }
};

Tensor rope_table_(const Tensor &inv_freq, int64_t n_pos, double scale, const OptTensor &out_,
                   const py::object &stream)
{
    gpu(inv_freq, "inv_freq", 1);
    typed(inv_freq, "inv_freq", at::kDouble);
    const int64_t n = inv_freq.size(0);
    if (n > 1 && inv_freq.stride(0) != 1)
        bad_value("inv_freq must be contiguous");
    if (n_pos < 0)
        bad_value("n_pos must not be negative");
    const On on(stream, inv_freq.get_device());
    const Tensor out = out_ ? *out_ : on.empty({n_pos, n, 2}, at::kFloat, inv_freq);
    const Angles a(out, inv_freq.get_device());
    if (a.n_pos != n_pos || a.n_freq != n)
        bad_value("out must be [n_pos, n_freq, 2]");
    done("rope_table",
         rope_table(static_cast<double *>(inv_freq.data_ptr()), a.p, n_pos, to_int32(n, "n_freq"),
                    scale, on.p));
    return out;
}

Tensor rope_(const Tensor &x, const Tensor &table, const Tensor &positions, bool interleaved,
             bool inverse, const OptTensor &out_, const py::object &out_dtype,
             const py::object &stream)
{
    heads(x, "x");
    const int dev = x.get_device();
    const auto want = dtype_of(out_dtype);
    const On on(stream, dev);
    const Tensor out = out_ ? *out_ : on.empty(x.sizes(), want.value_or(x.scalar_type()), x);
    if (out_) {
        heads(out, "out", dev);
        if (want)
            typed(out, "out", *want);
        if (out.sizes() != x.sizes())
            bad_value("out differs from x in shape");
    }
    const Angles a(table, dev);
    const int64_t T = x.size(0);
    const int32_t *pos = ints(positions, "positions", T, dev);
    const int in = code_of(x.scalar_type()), to = code_of(out.scalar_type());
    if (T)
        done("rope",
             rope(x.data_ptr(), x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
                  out.stride(1), pos, a.p, T, to_int32(x.size(1), "x"), to_int32(x.size(2), "x"),
                  a.n_pos, to_int32(a.n_freq, "table"), interleaved, inverse, in, to, on.p));
    return out;
}

OptTensor rope_kv_append_(const OptTensor &q, const Tensor &k, const Tensor &v,
                          const KvCache &cache, const KvBatch &batch, const Tensor &table,
                          const OptTensor &positions, bool interleaved, const OptTensor &q_out,
                          const py::object &stream)
{
    const int dev = cache.dev;
    heads(k, "k", dev);
    heads(v, "v", dev);
    typed(v, "v", k.scalar_type());
    const int64_t T = k.size(0), H = cache.c.n_heads, D = cache.c.head_dim;
    if (k.size(1) != H || k.size(2) != D || v.sizes() != k.sizes())
        bad_value("k and v must be [total_q, " + std::to_string(H) + ", " + std::to_string(D) + "]");
    auto even = [&](const Tensor &t) {
        return (t.size(1) <= 1 || t.stride(1) == D) && (T <= 1 || t.stride(0) == k.stride(0));
    };
    bool same = even(k) && even(v);
    const On on(stream, dev);
    OptTensor out;
    if (q) {
        heads(*q, "q", dev);
        typed(*q, "q", k.scalar_type());
        if (q->size(0) != T || q->size(2) != D)
            bad_value("q must be [total_q, n_q_heads, head_dim] of k's tokens and values");
        same = same && even(*q);
        out = q_out ? *q_out : on.empty(q->sizes(), cache.k.scalar_type(), cache.k);
        if (q_out) {
            gpu(*out, "q_out", 3, dev);
            typed(*out, "q_out", cache.k.scalar_type());
            if (out->sizes() != q->sizes() || !out->is_contiguous())
                bad_value("q_out must be contiguous, of q's shape");
        }
    }
    if (!same)
        bad_value("q, k and v need contiguous heads and the same stride between rows");
    const Angles a(table, dev);
    const int32_t *pos = positions ? ints(*positions, "positions", T, dev) : nullptr;
    const bqm_kv_batch b = batch.of(T, cache);
    const int in = code_of(k.scalar_type());
    if (T)
        done("rope_kv_append",
             rope_kv_append(q ? q->data_ptr() : nullptr, k.data_ptr(), v.data_ptr(), k.stride(0),
                            out ? out->data_ptr() : nullptr, &cache.c, &b, pos, a.p, a.n_pos,
                            to_int32(a.n_freq, "table"), interleaved,
                            q ? to_int32(q->size(1), "q") : 0, in, on.p));
    return out;
}

size_t paged_attention_workspace_bytes_(const KvCache &cache, const KvBatch &batch,
                                        int64_t n_q_heads, int64_t total_q)
{
    const bqm_kv_batch b = batch.of(total_q, cache);
    return paged_attention_workspace_bytes(&cache.c, &b, to_int32(n_q_heads, "n_q_heads"));
}

Tensor paged_attention_(const Tensor &q, const KvCache &cache, const KvBatch &batch,
                        std::optional<double> scale, bool causal, int64_t window,
                        const OptTensor &out_, const py::object &out_dtype,
                        const OptTensor &workspace, const py::object &stream)
{
    const int dev = cache.dev;
    heads(q, "q", dev);
    typed(q, "q", cache.k.scalar_type());
    const int64_t T = q.size(0), D = q.size(2);
    const int32_t H = to_int32(q.size(1), "q");
    if (D != cache.c.head_dim)
        bad_value("q has heads of " + std::to_string(D) + " values, the cache of " +
                  std::to_string(cache.c.head_dim));
    const auto want = dtype_of(out_dtype);
    const On on(stream, dev);
    const Tensor out = out_ ? *out_ : on.empty(q.sizes(), want.value_or(q.scalar_type()), q);
    if (out_) {
        gpu(out, "out", 3, dev);
        if (want)
            typed(out, "out", *want);
        if (out.sizes() != q.sizes() || !out.is_contiguous())
            bad_value("out must be contiguous, of q's shape");
    }
    const bqm_kv_batch b = batch.of(T, cache);
    const int to = code_of(out.scalar_type());
    if (T) {
        const Scratch w(workspace, paged_attention_workspace_bytes(&cache.c, &b, H), q, on);
        done("paged_attention",
             paged_attention(q.data_ptr(), q.stride(0), q.stride(1), &cache.c, &b, out.data_ptr(),
                             H, (float)scale.value_or(1.0 / std::sqrt((double)D)), causal,
                             to_int32(window, "window"), to, w.p, w.bytes, on.p));
    }
    return out;
}

// KvPages is a named tuple of the package's.
struct PagesArg {
    Tensor table, lens, refs;
    bqm_kv_pages p;
    int dev;

    PagesArg(const Tensor &t, const Tensor &l, const Tensor &r, const char *name, int on = -1)
        : table(t), lens(l), refs(r)
    {
        gpu(table, name, 2, on);
        typed(table, name, at::kInt);
        dev = table.get_device();
        if (table.size(1) > 1 && table.stride(1) != 1)
            bad_value("the table's rows must be contiguous");
        gpu(refs, "refs", 1, dev);
        p = {static_cast<int32_t *>(table.data_ptr()), ints(lens, "lens", table.size(0), dev),
             ints(refs, "refs", refs.size(0), dev), table.stride(0), refs.size(0),
             to_int32(table.size(0), name), to_int32(table.size(1), name)};
    }

    static PagesArg from(const py::object &o, const char *name, int on = -1)
    {
        Tensor t[3];
        if (!PyTuple_Check(o.ptr()) || PyTuple_GET_SIZE(o.ptr()) != 3)
            bad_type(text(name, " must be a KvPages"));
        for (int i = 0; i < 3; i++) {
            PyObject *x = PyTuple_GET_ITEM(o.ptr(), i);
            if (!THPVariable_Check(x))
                bad_type(text(name, " must hold GPU tensors"));
            t[i] = THPVariable_Unpack(x);
        }
        return PagesArg(t[0], t[1], t[2], name, on);
    }
};

// The state read and the one written.
struct InOut {
    PagesArg in;
    On on;
    PagesArg out;
    py::object result;

    static PagesArg out_of(const PagesArg &in, const py::object &given, const On &on)
    {
        if (!given.is_none()) {
            PagesArg o = PagesArg::from(given, "out", in.dev);
            if (o.table.sizes() != in.table.sizes() || o.refs.sizes() != in.refs.sizes())
                bad_value("out differs from pages in its sizes");
            return o;
        }
        return PagesArg(on.empty(in.table.sizes(), at::kInt, in.table),
                        on.empty(in.lens.sizes(), at::kInt, in.lens),
                        on.empty(in.refs.sizes(), at::kInt, in.refs), "out");
    }

    InOut(const py::object &pages, const py::object &given, const py::object &stream)
        : in(PagesArg::from(pages, "pages")), on(stream, in.dev), out(out_of(in, given, on)),
          result(given)
    {
        if (given.is_none())
            result = py::reinterpret_borrow<py::object>(g_pages)(out.table, out.lens, out.refs);
    }
};

py::tuple kv_extend_(const py::object &pages, const Tensor &n_new, int64_t page_size,
                     const py::object &out, const OptTensor &workspace, const py::object &stream)
{
    InOut s(pages, out, stream);
    const Tensor short_of = s.on.empty({1}, at::kInt, s.in.lens);
    const Scratch w(workspace, kv_pages_workspace_bytes(&s.in.p), s.in.lens, s.on);
    done("kv_extend",
         kv_extend(&s.in.p, &s.out.p, ints(n_new, "n_new", s.in.p.n_seqs, s.in.dev),
                   to_int32(page_size, "page_size"), static_cast<int32_t *>(short_of.data_ptr()),
                   w.p, w.bytes, s.on.p));
    return py::make_tuple(s.result, short_of);
}

py::tuple kv_fork_(const py::object &pages, const Tensor &parents, const Tensor &children,
                   int64_t page_size, const py::object &out, const OptTensor &workspace,
                   const py::object &stream)
{
    InOut s(pages, out, stream);
    gpu(parents, "parents", 1, s.in.dev);
    const int64_t n = parents.size(0);
    const Tensor moves = s.on.empty({n, 3}, at::kInt, s.in.lens);
    const Tensor short_of = s.on.empty({1}, at::kInt, s.in.lens);
    const Scratch w(workspace, kv_pages_workspace_bytes(&s.in.p), s.in.lens, s.on);
    int32_t *one = static_cast<int32_t *>(short_of.data_ptr());
    // an empty array has no address: any other stands for it
    auto some = [&](void *p) { return p ? static_cast<int32_t *>(p) : one; };
    done("kv_fork",
         kv_fork(&s.in.p, &s.out.p, some(ints(parents, "parents", n, s.in.dev)),
                 some(ints(children, "children", n, s.in.dev)), to_int32(n, "parents"),
                 to_int32(page_size, "page_size"), some(moves.data_ptr()), one, w.p, w.bytes,
                 s.on.p));
    return py::make_tuple(s.result, moves, short_of);
}

py::object kv_free_(const py::object &pages, const Tensor &seqs, const py::object &out,
                    const py::object &stream)
{
    InOut s(pages, out, stream);
    gpu(seqs, "seqs", 1, s.in.dev);
    const int64_t n = seqs.size(0);
    const int32_t *p = ints(seqs, "seqs", n, s.in.dev);
    done("kv_free", kv_free(&s.in.p, &s.out.p, n ? p : s.in.p.lens, to_int32(n, "seqs"),
                            s.on.p));
    return s.result;
}

py::tuple kv_compact_(const py::object &pages, int64_t page_size, const py::object &out,
                      const py::object &stream)
{
    InOut s(pages, out, stream);
    const Tensor moves = s.on.empty({s.in.p.n_pages / 2, 3}, at::kInt, s.in.lens);
    const Tensor page_map = s.on.empty({s.in.p.n_pages}, at::kInt, s.in.lens);
    int32_t *map = static_cast<int32_t *>(page_map.data_ptr());
    int32_t *m = moves.numel() ? static_cast<int32_t *>(moves.data_ptr()) : map;
    done("kv_compact", kv_compact(&s.in.p, &s.out.p, to_int32(page_size, "page_size"), map, m,
                                  s.on.p));
    return py::make_tuple(s.result, moves, page_map);
}

void kv_copy_pages_(const KvCache &cache, const Tensor &moves, const py::object &stream)
{
    gpu(moves, "moves", 2, cache.dev);
    typed(moves, "moves", at::kInt);
    if (moves.size(1) != 3 || !moves.is_contiguous())
        bad_value("moves must be contiguous [n, 3]");
    if (moves.size(0)) {
        const On on(stream, cache.dev);
        done("kv_copy_pages", kv_copy_pages(&cache.c, static_cast<int32_t *>(moves.data_ptr()),
                                            moves.size(0), on.p));
    }
}

}  // namespace

PYBIND11_MODULE(_attention, m)
{
    const py::arg_v stream("stream", py::none()), out("out", py::none());
    const py::arg_v workspace("workspace", py::none()), dtype("out_dtype", py::none());
    m.def("set_python", &set_python);
    py::class_<KvCache>(m, "KvCache",
                        "Keys and values in pages: two tensors [n_pages, page_size, n_heads, head_dim], "
                        "or with the\nlayers of a model before the pages, float16 or bfloat16, of the same "
                        "strides; any order of pages,\ntokens and heads in memory, a head's values "
                        "contiguous.")
        .def(py::init<const Tensor &, const Tensor &>(), py::arg("k"), py::arg("v"))
        .def_readonly("k", &KvCache::k)
        .def_readonly("v", &KvCache::v)
        .def_property_readonly("n_layers", [](const KvCache &c) { return c.c.n_layers; })
        .def_property_readonly("n_pages", [](const KvCache &c) { return c.c.n_pages; })
        .def_property_readonly("page_size", [](const KvCache &c) { return c.c.page_size; })
        .def_property_readonly("n_heads", [](const KvCache &c) { return c.c.n_heads; })
        .def_property_readonly("head_dim", [](const KvCache &c) { return c.c.head_dim; })
        .def("layer", &KvCache::layer, py::arg("i"),
             "The cache of layer i alone (the one attention and the append use).");
    py::class_<KvBatch>(m, "KvBatch",
                        "The new tokens of a step: table int32 [n_seqs, max_pages], kv_lens int32 [n_seqs] "
                        "(the new tokens\ncounted), q_starts int32 [n_seqs + 1]. max_q and max_kv bound the "
                        "sequences' new tokens and tokens on\nthe host (by default whatever the arrays could "
                        "hold; closer bounds give better launches).")
        .def(py::init<const Tensor &, const Tensor &, const Tensor &, std::optional<int64_t>,
                      std::optional<int64_t>>(),
             py::arg("table"), py::arg("kv_lens"), py::arg("q_starts"),
             py::arg("max_q") = py::none(), py::arg("max_kv") = py::none())
        .def_readonly("table", &KvBatch::table)
        .def_readonly("kv_lens", &KvBatch::kv_lens)
        .def_readonly("q_starts", &KvBatch::q_starts);
    m.def("rope_table", &rope_table_, py::arg("inv_freq"), py::arg("n_pos"),
          py::arg("scale") = 1.0, out, stream,
          "(cos, sin) of position * inv_freq times scale: fp32 [n_pos, n_freq, 2].");
    m.def("rope", &rope_, py::arg("x"), py::arg("table"), py::arg("positions"),
          py::arg("interleaved") = false, py::arg("inverse") = false, out, dtype, stream,
          "x [T, n_heads, head_dim] (any strides, values contiguous) turned by the angles of table "
          "(rope_table) at\npositions int32 [T]; inverse turns back (the gradient). out may be x itself.");
    m.def("rope_kv_append", &rope_kv_append_, py::arg("q"), py::arg("k"), py::arg("v"),
          py::arg("cache"), py::arg("batch"), py::arg("table"), py::arg("positions") = py::none(),
          py::arg("interleaved") = false, py::arg("q_out") = py::none(), stream,
          "Turns q [total_q, n_q_heads, head_dim] into q_out (of the cache's type) and k [total_q, n_heads, "
          "head_dim]\ninto the cache, and stores v there, at the new tokens' places. q, k and v may be slices "
          "of one product's\nrows (one stride between rows, heads contiguous); q may be None.");
    m.def("paged_attention_workspace_bytes", &paged_attention_workspace_bytes_, py::arg("cache"),
          py::arg("batch"), py::arg("n_q_heads"), py::arg("total_q"));
    m.def("paged_attention", &paged_attention_, py::arg("q"), py::arg("cache"), py::arg("batch"),
          py::arg("scale") = py::none(), py::arg("causal") = true, py::arg("window") = 0, out,
          dtype, workspace, stream,
          "Attention of q [total_q, n_q_heads, head_dim] (the cache's type; strides of multiples of 8) over "
          "the batch's\npages of the cache; scale defaults to head_dim ** -0.5, window 0 is none. out is "
          "contiguous, of the cache's\ntype or float32; rows that see no token are zeros.");
    m.def("kv_extend", &kv_extend_, py::arg("pages"), py::arg("n_new"), py::arg("page_size"), out,
          workspace, stream,
          "Room for n_new int32 [n_seqs] more tokens: (pages, short_of), short_of int32 [1] on the GPU the "
          "count of\nsequences that got none. out: where the new state goes (pages itself: in place).");
    m.def("kv_fork", &kv_fork_, py::arg("pages"), py::arg("parents"), py::arg("children"),
          py::arg("page_size"), out, workspace, stream,
          "Row children[i] becomes a fork of row parents[i] (int32 [n] both): (pages, moves, short_of), moves "
          "int32\n[n, 3] for kv_copy_pages, short_of as for kv_extend.");
    m.def("kv_free", &kv_free_, py::arg("pages"), py::arg("seqs"), out, stream,
          "The rows seqs int32 [n] end and give their pages back.");
    m.def("kv_compact", &kv_compact_, py::arg("pages"), py::arg("page_size"), out, stream,
          "Used pages move into the free ones before them: (pages, moves, page_map), moves int32 "
          "[n_pages // 2, 3] for\nkv_copy_pages, page_map int32 [n_pages] where each page's tokens are now.");
    m.def("kv_copy_pages", &kv_copy_pages_, py::arg("cache"), py::arg("moves"), stream,
          "Copies moves int32 [n, 3] = (from page, to page, tokens) in every layer.");
}
