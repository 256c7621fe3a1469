// rope.hip -- rotary positions: the table of angles, the rotation of a tensor
// of heads, and the rotation of new queries and keys together with the store
// of keys and values into the pages of a cache.
//
// A pair (x_a, x_b) turns by (c, s): y_a = x_a c - x_b s, y_b = x_b c + x_a s,
// in fp32 with one rounding to the output's type. Three operations and two
// angles (shared by all heads of a token) for two values read and written:
// memory bounds it at every size above a launch: 8191 tokens of 48 heads of 128,
// bf16, appended in 46 us (4.5 TB/s), 4099 x 32 heads of 96 turned in 12 us
// (4.3 TB/s), 33 tokens in 3.5 us. Loads or stores past the caches, and workgroups
// of 128, measured no faster.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }

// Eight values, as one thread's 16 or 32 bytes.
template <class T>
struct Eight {
    T v[8];
};

template <class T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8])
{
    Eight<T> e;
    if constexpr (sizeof(T) == 2) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        __builtin_memcpy(&e, &r, 16);
    } else {
        const uint4 r = reinterpret_cast<const uint4 *>(p)[0];
        const uint4 s = reinterpret_cast<const uint4 *>(p)[1];
        __builtin_memcpy(&e, &r, 16);
        __builtin_memcpy(e.v + 4, &s, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        x[i] = to_f32(e.v[i]);
}

template <class T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8])
{
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < 8; i++)
        e.v[i] = (T)x[i];
    if constexpr (sizeof(T) == 2) {
        uint4 r;
        __builtin_memcpy(&r, &e, 16);
        *reinterpret_cast<uint4 *>(p) = r;
    } else {
        uint4 r, s;
        __builtin_memcpy(&r, &e, 16);
        __builtin_memcpy(&s, e.v + 4, 16);
        reinterpret_cast<uint4 *>(p)[0] = r;
        reinterpret_cast<uint4 *>(p)[1] = s;
    }
}

// How a head's values are dealt to threads: `pairs` units that turn, then
// `rest` units that copy. A unit is, with VEC, eight values (interleaved: four
// pairs) or eight pairs (halves: eight values at i and their eight partners
// at n_freq + i); without, one pair or one value.
struct Head {
    int dim, n_freq, pairs, rest;
    bool interleaved;
    float sign;  // of the sine
};

Head head_of(int dim, int n_freq, bool interleaved, bool inverse, bool vec)
{
    Head h = {dim, n_freq, 0, 0, interleaved, inverse ? -1.0f : 1.0f};
    h.pairs = vec ? n_freq / (interleaved ? 4 : 8) : n_freq;
    h.rest = vec ? (dim - 2 * n_freq) / 8 : dim - 2 * n_freq;
    return h;
}

// Whether a head can be dealt in eights: no unit straddles the halves or the end.
bool deals_in_eights(int dim, int n_freq, bool interleaved)
{
    return dim % 8 == 0 && n_freq % (interleaved ? 4 : 8) == 0;
}

template <bool VEC, class TI, class TO>
__device__ __forceinline__ void copy_unit(const TI *x, TO *y, int u)
{
    if constexpr (VEC) {
        float a[8];
        load8(x + 8 * u, a);
        store8(y + 8 * u, a);
    } else {
        y[u] = (TO)to_f32(x[u]);
    }
}

// Unit u of a head at x, to the same unit at y (which may be x).
template <bool VEC, class TI, class TO>
__device__ __forceinline__ void turn_unit(const Head &h, const TI *x, TO *y, const float2 *cs,
                                          int u)
{
    if (u >= h.pairs) {
        copy_unit<VEC>(x + 2 * h.n_freq, y + 2 * h.n_freq, u - h.pairs);
        return;
    }
    if constexpr (!VEC) {
        const int a = h.interleaved ? 2 * u : u, b = h.interleaved ? 2 * u + 1 : u + h.n_freq;
        const float2 t = cs[u];
        const float xa = to_f32(x[a]), xb = to_f32(x[b]), s = t.y * h.sign;
        y[a] = (TO)(xa * t.x - xb * s);
        y[b] = (TO)(xb * t.x + xa * s);
    } else if (h.interleaved) {
        float v[8], w[8];
        load8(x + 8 * u, v);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 t = cs[4 * u + i];
            const float s = t.y * h.sign;
            w[2 * i] = v[2 * i] * t.x - v[2 * i + 1] * s;
            w[2 * i + 1] = v[2 * i + 1] * t.x + v[2 * i] * s;
        }
        store8(y + 8 * u, w);
    } else {
        float a[8], b[8], p[8], q[8];
        load8(x + 8 * u, a);
        load8(x + h.n_freq + 8 * u, b);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 t = cs[8 * u + i];
            const float s = t.y * h.sign;
            p[i] = a[i] * t.x - b[i] * s;
            q[i] = b[i] * t.x + a[i] * s;
        }
        store8(y + 8 * u, p);
        store8(y + h.n_freq + 8 * u, q);
    }
}

__global__ __launch_bounds__(256) void rope_table_kernel(const double *inv_freq, float2 *table,
                                                         int64_t n, int n_freq, double scale)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256) {
        double s, c;
        sincos((double)(i / n_freq) * inv_freq[i % n_freq], &s, &c);
        table[i] = make_float2((float)(scale * c), (float)(scale * s));
    }
}

__device__ __forceinline__ const float2 *row_of(const float2 *table, int pos, int64_t n_pos,
                                                int n_freq)
{
    const int64_t p = pos < 0 ? 0 : (pos < n_pos ? pos : n_pos - 1);
    return table + p * n_freq;
}

struct RopeArgs {
    const void *x;
    void *y;
    int64_t x_token, x_head, y_token, y_head;
    const int32_t *positions;
    const float2 *table;
    int64_t n_pos;
    int64_t units;  // of one token
    Head head;
};

// Block (token, piece of its units); the token's row of angles is uniform.
template <class TI, class TO, bool VEC>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a)
{
    const int64_t t = blockIdx.x;
    const int i = blockIdx.y * 256 + threadIdx.x;
    if (i >= a.units)
        return;
    const int per = a.head.pairs + a.head.rest, h = i / per;
    turn_unit<VEC>(a.head, static_cast<const TI *>(a.x) + t * a.x_token + h * a.x_head,
                   static_cast<TO *>(a.y) + t * a.y_token + h * a.y_head,
                   row_of(a.table, a.positions[t], a.n_pos, a.head.n_freq), i - h * per);
}

struct AppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    int64_t token;                         // stride of q, k and v
    int64_t c_page, c_token, c_head;       // strides of the cache
    const int32_t *pages, *kv_lens, *q_starts, *positions;
    int64_t pages_stride;
    const float2 *table;
    int64_t n_pos;
    int64_t total_q, n_pages;
    int n_seqs, max_pages, page_size, n_q_heads, n_heads;
    int q_units, k_units, v_units;         // of one token
    Head head;
};

// The sequence of row t: the last b with q_starts[b] <= t.
__device__ __forceinline__ int sequence_of(const int32_t *q_starts, int n_seqs, int64_t t)
{
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q_starts[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <class TI, class TO, bool VEC>
__global__ __launch_bounds__(256) void rope_append_kernel(AppendArgs a)
{
    const int64_t t = blockIdx.x;
    int i = blockIdx.y * 256 + threadIdx.x;
    const int b = sequence_of(a.q_starts, a.n_seqs, t);
    const int64_t place = (int64_t)a.kv_lens[b] - a.q_starts[b + 1] + t;
    const int pos = a.positions ? a.positions[t] : (int)place;
    const float2 *cs = row_of(a.table, pos, a.n_pos, a.head.n_freq);
    const int per = a.head.pairs + a.head.rest;
    if (i < a.q_units) {
        const int h = i / per;
        turn_unit<VEC>(a.head, static_cast<const TI *>(a.q) + t * a.token + (int64_t)h * a.head.dim,
                       static_cast<TO *>(a.q_out) +
                           (t * a.n_q_heads + h) * (int64_t)a.head.dim,
                       cs, i - h * per);
        return;
    }
    i -= a.q_units;
    if (place < 0 || place >= (int64_t)a.max_pages * a.page_size)
        return;
    const int page = a.pages[b * a.pages_stride + place / a.page_size];
    if ((uint64_t)(int64_t)page >= (uint64_t)a.n_pages)
        return;
    const int64_t at = page * a.c_page + (place % a.page_size) * a.c_token;
    if (i < a.k_units) {
        const int h = i / per;
        turn_unit<VEC>(a.head, static_cast<const TI *>(a.k) + t * a.token + (int64_t)h * a.head.dim,
                       static_cast<TO *>(a.k_cache) + at + h * a.c_head, cs, i - h * per);
        return;
    }
    i -= a.k_units;
    if (i < a.v_units) {
        const int n = VEC ? a.head.dim / 8 : a.head.dim, h = i / n;
        copy_unit<VEC>(static_cast<const TI *>(a.v) + t * a.token + (int64_t)h * a.head.dim,
                       static_cast<TO *>(a.v_cache) + at + h * a.c_head, i - h * n);
    }
}

// f(in, out, vec) with values whose types are the tensors' element types.
template <class F>
int with_types(int in, int out, bool vec, F f)
{
    auto with_out = [&](auto ti) {
        auto with_vec = [&](auto to) {
            return vec ? f(ti, to, std::true_type{}) : f(ti, to, std::false_type{});
        };
        if (out == BQM_DTYPE_F32)
            return with_vec(float{});
        return out == BQM_DTYPE_F16 ? with_vec(_Float16{}) : with_vec(__bf16{});
    };
    if (in == BQM_DTYPE_F32)
        return with_out(float{});
    return in == BQM_DTYPE_F16 ? with_out(_Float16{}) : with_out(__bf16{});
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
int64_t bytes_of(int dtype) { return dtype == BQM_DTYPE_F32 ? 4 : 2; }

// Whether rows `a` and `b` elements apart keep 16-byte alignment.
bool strides16(int64_t a, int64_t b, int dtype)
{
    return (a | b) * bytes_of(dtype) % 16 == 0;
}

}  // namespace

int launch_rope_table(const double *inv_freq, float *table, int64_t n_pos, int n_freq,
                      double scale, hipStream_t stream)
{
    const int64_t n = n_pos * n_freq;
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 65536)),
                       dim3(256), 0, stream, inv_freq, reinterpret_cast<float2 *>(table), n,
                       n_freq, scale);
    return check_launch();
}

int launch_rope(const void *x, int64_t x_token, int64_t x_head, void *y, int64_t y_token,
                int64_t y_head, const int32_t *positions, const float *table, int64_t T,
                int n_heads, int head_dim, int64_t n_pos, int n_freq, bool interleaved,
                bool inverse, int in_dtype, int out_dtype, hipStream_t stream)
{
    const bool vec = deals_in_eights(head_dim, n_freq, interleaved) && aligned16(x) &&
                     aligned16(y) && strides16(x_token, x_head, in_dtype) &&
                     strides16(y_token, y_head, out_dtype);
    const Head head = head_of(head_dim, n_freq, interleaved, inverse, vec);
    const int64_t units = (int64_t)n_heads * (head.pairs + head.rest);
    const RopeArgs a = {x,         y,     x_token, x_head, y_token, y_head,
                        positions, reinterpret_cast<const float2 *>(table), n_pos, units, head};
    return with_types(in_dtype, out_dtype, vec, [&](auto ti, auto to, auto v) {
        hipLaunchKernelGGL((rope_kernel<decltype(ti), decltype(to), decltype(v)::value>),
                           dim3((unsigned)T, (unsigned)((units + 255) / 256)), dim3(256), 0,
                           stream, a);
        return check_launch();
    });
}

int launch_rope_append(const void *q, const void *k, const void *v, int64_t token_stride,
                       void *q_out, const bqm_kv_cache *c, const bqm_kv_batch *b,
                       const int32_t *positions, const float *table, int64_t n_pos, int n_freq,
                       bool interleaved, int n_q_heads, int in_dtype, hipStream_t stream)
{
    const int dim = c->head_dim;
    const bool vec = deals_in_eights(dim, n_freq, interleaved) && (!q || aligned16(q)) &&
                     aligned16(k) && aligned16(v) && strides16(token_stride, dim, in_dtype);
    const Head head = head_of(dim, n_freq, interleaved, false, vec);
    const int per = head.pairs + head.rest;
    AppendArgs a = {q, k, v, q_out, c->k, c->v, token_stride,
                    c->page_stride, c->token_stride, c->head_stride,
                    b->table, b->kv_lens, b->q_starts, positions, b->table_stride,
                    reinterpret_cast<const float2 *>(table), n_pos, b->total_q, c->n_pages,
                    b->n_seqs, b->max_pages, c->page_size, n_q_heads, c->n_heads,
                    n_q_heads * per, c->n_heads * per, c->n_heads * (vec ? dim / 8 : dim), head};
    const int64_t units = (int64_t)a.q_units + a.k_units + a.v_units;
    const dim3 grid((unsigned)b->total_q, (unsigned)((units + 255) / 256));
    return with_types(in_dtype, c->dtype, vec, [&](auto ti, auto to, auto vv) {
        if constexpr (sizeof(to) == 2)
            hipLaunchKernelGGL((rope_append_kernel<decltype(ti), decltype(to), decltype(vv)::value>),
                               grid, dim3(256), 0, stream, a);
        return check_launch();
    });
}

}  // namespace bqm
