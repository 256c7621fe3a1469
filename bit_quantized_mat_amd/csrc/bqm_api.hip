// bqm_api.hip -- the C ABI declared in include/bqm.h: argument validation on
// the host, one dispatch point per entry, launches on the caller's stream.
#include <math.h>
#include <string.h>

#include <atomic>

#include "common.hpp"
#include "launch.hpp"

namespace {

constexpr int kVersion = 200;  // 0.2.0
constexpr uint64_t kMaxBufferBytes = 0xfffffffcull;  // 32-bit byte offsets inside one matrix

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// Device check, cached per device ordinal: gfx950 only.
int check_device()
{
    // 0 unknown, 1 ok, -1 not gfx950; atomics, so concurrent first calls
    // from several host threads each store the same value without a race
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return BQM_ERR_DEVICE;
    if (dev < 64) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c)
            return c > 0 ? BQM_OK : BQM_ERR_DEVICE;
    }
    hipDeviceProp_t prop;
    int ok = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
             strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64)
        cached[dev].store(ok ? 1 : -1, std::memory_order_relaxed);
    return ok ? BQM_OK : BQM_ERR_DEVICE;
}

hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

// block_bytes: 54 for TQ1_0, 66 for TQ2_0
int check_matrix(int64_t N, int64_t K, uint64_t block_bytes = 54)
{
    if (N < 1 || K < 256 || K % 256 != 0)
        return BQM_ERR_SHAPE;
    if ((uint64_t)N * (uint64_t)(K / 256) * block_bytes > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    return BQM_OK;
}

}  // namespace

extern "C" {

int tq1_pack(const int8_t *trits, const uint16_t *d, void *w, int64_t N, int64_t K,
             void *stream)
{
    if (!trits || !d || !w)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K))
        return rc;
    if (int rc = check_device())
        return rc;
    return bqm::launch_tq1_pack(trits, d, w, N, K, as_stream(stream));
}

int q8_1_quantize(const float *x, void *a, int64_t T, int64_t K, void *stream)
{
    if (!x || !a)
        return BQM_ERR_NULL;
    if (T < 1 || K < 32 || K % 32 != 0 || (uint64_t)T * (uint64_t)K > (1ull << 40))
        return BQM_ERR_SHAPE;
    if (!aligned4(x) || !aligned4(a))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_q8_1_quantize(x, a, T, K, as_stream(stream));
}

// The residual must be the output itself or lie wholly outside it: each
// output element is read from r and written to y by the same lane, so only
// a partial overlap could mix elements.
static bool residual_ok(const float *r, const void *y, int64_t N, int32_t T)
{
    if ((const void *)r == y)
        return true;
    const uintptr_t rb = (uintptr_t)r, yb = (uintptr_t)y, n = (uintptr_t)N * (uintptr_t)T * 4u;
    return rb + n <= yb || yb + n <= rb;
}

// r: the residual of the add entry point (nullptr for the others);
// block_bytes: the weight format's block size.
static int mmvq_common(const void *w, const void *a, const void *out, int64_t N, int64_t K,
                       int32_t T, const float *r = nullptr, uint64_t block_bytes = 54)
{
    if (!w || !a || !out)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K, block_bytes))
        return rc;
    if (T < 1 || T > BQM_MMVQ_MAX_COLS)
        return BQM_ERR_SHAPE;
    if ((uint64_t)T * (uint64_t)(K / 32) * 36ull > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (r && !residual_ok(r, out, N, T))
        return BQM_ERR_SHAPE;
    if (!aligned4(w) || !aligned4(a) || !aligned4(out) || (r && !aligned4(r)))
        return BQM_ERR_ALIGN;
    return check_device();
}

int mmvq_tq1_0(const void *w, const void *a, float *y, int64_t N, int64_t K, int32_t T,
               void *stream)
{
    if (int rc = mmvq_common(w, a, y, N, K, T))
        return rc;
    return bqm::launch_mmvq(w, a, y, nullptr, N, K, T, as_stream(stream));
}

int mmvq_tq1_0_add(const void *w, const void *a, const float *r, float *y, int64_t N, int64_t K,
                   int32_t T, void *stream)
{
    if (!r)
        return BQM_ERR_NULL;
    if (int rc = mmvq_common(w, a, y, N, K, T, r))
        return rc;
    return bqm::launch_mmvq(w, a, y, nullptr, N, K, T, as_stream(stream), r);
}

int mm_tq1_0(const void *w, const void *a, float *y, int64_t N, int64_t K, int64_t T,
             void *stream)
{
    if (!w || !a || !y)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K))
        return rc;
    if (T < 1 || T > BQM_MM_MAX_COLS || (uint64_t)T * (uint64_t)(K / 32) * 36ull > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (!aligned4(w) || !aligned4(a) || !aligned4(y))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_mm(w, a, y, N, K, T, as_stream(stream));
}

// with_r: the residual-add entry point (r required).
static int mmvq_f32_call(const void *w, const float *x, const float *r, bool with_r, float *y,
                         int64_t N, int64_t K, int32_t T, void *stream)
{
    if (!w || !x || !y || (with_r && !r))
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K))
        return rc;
    if (T < 1 || T > BQM_MMVQ_F32_MAX_COLS || (uint64_t)T * (uint64_t)K * 4ull > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (with_r && !residual_ok(r, y, N, T))
        return BQM_ERR_SHAPE;
    if (!aligned4(w) || !aligned4(x) || !aligned4(y) || (with_r && !aligned4(r)))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    // three to eight columns: the quad kernel where it takes the shape (it
    // stages, and so quantizes, each column once per 16 rows like the staged
    // kernel, with a quarter of the staged kernel's LDS reads)
    if (bqm::quad_supported(K, T))
        return bqm::launch_mmvq_quad_f32(w, x, y, N, K, T, as_stream(stream), r);
    if (!bqm::staged_supported(K, T))
        return BQM_ERR_SHAPE;
    return bqm::launch_mmvq_staged_f32(w, x, y, N, K, T, as_stream(stream), r);
}

int mmvq_tq1_0_f32(const void *w, const float *x, float *y, int64_t N, int64_t K, int32_t T,
                   void *stream)
{
    return mmvq_f32_call(w, x, nullptr, false, y, N, K, T, stream);
}

int mmvq_tq1_0_f32_add(const void *w, const float *x, const float *r, float *y, int64_t N,
                       int64_t K, int32_t T, void *stream)
{
    return mmvq_f32_call(w, x, r, true, y, N, K, T, stream);
}

// f32: the columns are fp32 (quantized inside the call, at most two), else
// Q8_1 blocks. Up to two columns one launch of the staged wave pairs; beyond,
// the gate product into y, then the up product with the gated epilogue
// reading y.
static int glu_call(const void *wg, const void *wu, const void *a, float *y, int64_t N,
                    int64_t K, int32_t T, bool f32, void *stream)
{
    if (!wg || !wu || !a || !y)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K))
        return rc;
    const uint64_t col_bytes = f32 ? (uint64_t)K * 4ull : (uint64_t)(K / 32) * 36ull;
    const int max_cols = f32 ? BQM_GLU_F32_MAX_COLS : BQM_GLU_MAX_COLS;
    if (T < 1 || T > max_cols || (uint64_t)T * col_bytes > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (!aligned4(wg) || !aligned4(wu) || !aligned4(a) || !aligned4(y))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    const hipStream_t st = as_stream(stream);
    if (T <= bqm::kGluMaxCols)
        return bqm::launch_mmvq_glu(wg, wu, a, y, N, K, T, f32, st);
    if (int rc = bqm::launch_mmvq(wg, a, y, nullptr, N, K, T, st))
        return rc;
    return bqm::launch_mmvq(wu, a, y, nullptr, N, K, T, st, bqm::gated_epilogue(y));
}

int mmvq_tq1_0_glu(const void *w_gate, const void *w_up, const void *a, float *y, int64_t N,
                   int64_t K, int32_t T, void *stream)
{
    return glu_call(w_gate, w_up, a, y, N, K, T, false, stream);
}

int mmvq_tq1_0_f32_glu(const void *w_gate, const void *w_up, const float *x, float *y,
                       int64_t N, int64_t K, int32_t T, void *stream)
{
    return glu_call(w_gate, w_up, x, y, N, K, T, true, stream);
}

int mmvq_tq1_0_block_isums(const void *w, const void *a, int32_t *isums, int64_t N, int64_t K,
                           int32_t T, void *stream)
{
    if (int rc = mmvq_common(w, a, isums, N, K, T))
        return rc;
    return bqm::launch_mmvq(w, a, nullptr, isums, N, K, T, as_stream(stream));
}

int tq2_pack(const int8_t *trits, const uint16_t *d, void *w, int64_t N, int64_t K,
             void *stream)
{
    if (!trits || !d || !w)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K, 66))
        return rc;
    if (int rc = check_device())
        return rc;
    return bqm::launch_tq2_pack(trits, d, w, N, K, as_stream(stream));
}

int mmvq_tq2_0(const void *w, const void *a, float *y, int64_t N, int64_t K, int32_t T,
               void *stream)
{
    if (int rc = mmvq_common(w, a, y, N, K, T, nullptr, 66))
        return rc;
    return bqm::launch_mmvq_tq2(w, a, y, nullptr, N, K, T, as_stream(stream));
}

int mmvq_tq2_0_block_isums(const void *w, const void *a, int32_t *isums, int64_t N, int64_t K,
                           int32_t T, void *stream)
{
    if (int rc = mmvq_common(w, a, isums, N, K, T, nullptr, 66))
        return rc;
    return bqm::launch_mmvq_tq2(w, a, nullptr, isums, N, K, T, as_stream(stream));
}

int tq1_dequantize(const void *w, const int32_t *rows, void *out, int64_t N, int64_t K,
                   int64_t n_rows, int32_t out_dtype, void *stream)
{
    if (!w || !out)
        return BQM_ERR_NULL;
    if (int rc = check_matrix(N, K))
        return rc;
    if (n_rows < 1 || (!rows && n_rows > N) || n_rows * (K / 256) >= (1ll << 27) ||
        out_dtype < BQM_DTYPE_F32 || out_dtype > BQM_DTYPE_BF16)
        return BQM_ERR_SHAPE;
    // every dtype's kernel stores 16 bytes per lane
    if (!aligned4(w) || (rows && !aligned4(rows)) || ((uintptr_t)out & 15u))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_tq1_dequantize(w, rows, out, N, K, n_rows, out_dtype, as_stream(stream));
}

size_t mmvq_id_tq1_0_workspace_bytes(int64_t E, int64_t T, int32_t n_used)
{
    if (E < 1 || T < 1 || n_used < 1 || n_used > E || T * (int64_t)n_used > 65535)
        return 0;
    return bqm::mmvq_id_workspace_bytes(E, T, n_used);
}

// Both expert-routed products; per_slot: one activation column per
// (token, slot) pair instead of one per token.
static int mmvq_id_call(const void *w, const void *a, const int32_t *ids, float *y, int64_t E,
                        int64_t N, int64_t K, int64_t T, int32_t n_used, bool per_slot,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    if (!w || !a || !ids || !y)
        return BQM_ERR_NULL;
    if (E < 1 || T < 1 || n_used < 1 || n_used > E || T * (int64_t)n_used > 65535)
        return BQM_ERR_SHAPE;
    if (int rc = check_matrix(N, K))
        return rc;
    const uint64_t a_cols = (uint64_t)T * (per_slot ? (uint64_t)n_used : 1ull);
    if (a_cols * (uint64_t)(K / 32) * 36ull > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (!aligned4(w) || !aligned4(a) || !aligned4(ids) || !aligned4(y))
        return BQM_ERR_ALIGN;
    const size_t need = bqm::mmvq_id_workspace_bytes(E, T, n_used);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return BQM_ERR_WORKSPACE;
    if (workspace && ((uintptr_t)workspace & 255u) != 0)
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_mmvq_id(w, a, ids, y, E, N, K, T, n_used, per_slot, workspace,
                               as_stream(stream));
}

int mmvq_id_tq1_0(const void *w, const void *a, const int32_t *ids, float *y, int64_t E,
                  int64_t N, int64_t K, int64_t T, int32_t n_used, void *workspace,
                  size_t workspace_bytes, void *stream)
{
    return mmvq_id_call(w, a, ids, y, E, N, K, T, n_used, false, workspace, workspace_bytes,
                        stream);
}

int mmvq_id_tq1_0_noalloc(const void *w, const void *a, const int32_t *ids, float *y, int64_t E,
                          int64_t N, int64_t K, int64_t T, int32_t n_used, void *stream)
{
    // the same checks as mmvq_id_tq1_0, except that the workspace is the
    // library's device scratch
    if (!w || !a || !ids || !y)
        return BQM_ERR_NULL;
    if (E < 1 || T < 1 || n_used < 1 || n_used > E || T * (int64_t)n_used > 65535)
        return BQM_ERR_SHAPE;
    if (int rc = check_matrix(N, K))
        return rc;
    if ((uint64_t)T * (uint64_t)(K / 32) * 36ull > kMaxBufferBytes)
        return BQM_ERR_SHAPE;
    if (!aligned4(w) || !aligned4(a) || !aligned4(ids) || !aligned4(y))
        return BQM_ERR_ALIGN;
    if (bqm::mmvq_id_workspace_bytes(E, T, n_used) > bqm::kNoAllocScratchBytes)
        return BQM_ERR_WORKSPACE;
    if (int rc = check_device())
        return rc;
    void *scratch = nullptr;
    if (int rc = bqm::noalloc_scratch(&scratch))
        return rc;
    return bqm::launch_mmvq_id(w, a, ids, y, E, N, K, T, n_used, false, scratch,
                               as_stream(stream));
}

int mmvq_id_tq1_0_slots(const void *w, const void *a, const int32_t *ids, float *y, int64_t E,
                        int64_t N, int64_t K, int64_t T, int32_t n_used, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    return mmvq_id_call(w, a, ids, y, E, N, K, T, n_used, true, workspace, workspace_bytes,
                        stream);
}

// ---- attention side ----------------------------------------------------------

static bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
static bool is_dtype(int d) { return d >= BQM_DTYPE_F32 && d <= BQM_DTYPE_BF16; }
static uintptr_t bytes_of(int d) { return d == BQM_DTYPE_F32 ? 4 : 2; }

static int check_cache(const bqm_kv_cache *c)
{
    if (!c || !c->k || !c->v)
        return BQM_ERR_NULL;
    if (c->n_layers < 1 || c->n_layers > (1 << 20) || c->n_pages < 1 || c->n_pages > (1 << 30) ||
        c->page_size < 1 || c->page_size > 65536 || c->n_heads < 1 || c->n_heads > 65535 ||
        c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8 != 0 ||
        (c->dtype != BQM_DTYPE_F16 && c->dtype != BQM_DTYPE_BF16))
        return BQM_ERR_SHAPE;
    const int64_t most = 1ll << 35;
    for (const int64_t s : {c->page_stride, c->token_stride, c->head_stride, c->layer_stride})
        if (s < 0 || s > (1ll << 50))
            return BQM_ERR_SHAPE;
    // the kernels count 16-byte pieces of a layer in 32 bits
    const double span = (double)(c->n_pages - 1) * (double)c->page_stride +
                        (double)(c->page_size - 1) * (double)c->token_stride +
                        (double)(c->n_heads - 1) * (double)c->head_stride + c->head_dim;
    if (span >= (double)most)
        return BQM_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) ||
        (c->page_stride | c->token_stride | c->head_stride | c->layer_stride) % 8 != 0)
        return BQM_ERR_ALIGN;
    return BQM_OK;
}

static int check_batch(const bqm_kv_batch *b)
{
    if (!b || !b->table || !b->kv_lens || !b->q_starts)
        return BQM_ERR_NULL;
    if (b->n_seqs < 1 || b->n_seqs > 65535 || b->max_pages < 1 || b->max_pages > (1 << 24) ||
        b->table_stride < 0 || b->total_q < 0 || b->total_q > (1 << 23) || b->max_q < 0 ||
        b->max_kv < 0 || b->max_kv > (1 << 30))
        return BQM_ERR_SHAPE;
    if (!aligned4(b->table) || !aligned4(b->kv_lens) || !aligned4(b->q_starts))
        return BQM_ERR_ALIGN;
    return BQM_OK;
}

int rope_table(const double *inv_freq, float *table, int64_t n_pos, int32_t n_freq, double scale,
               void *stream)
{
    if (!inv_freq || !table)
        return BQM_ERR_NULL;
    if (n_pos < 1 || n_pos > 0x7fffffff || n_freq < 1 || n_freq > 512)
        return BQM_ERR_SHAPE;
    if (!aligned(inv_freq, 8) || !aligned(table, 8))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_rope_table(inv_freq, table, n_pos, n_freq, scale, as_stream(stream));
}

int rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y,
         int64_t y_token_stride, int64_t y_head_stride, const int32_t *positions,
         const float *table, int64_t T, int32_t n_heads, int32_t head_dim, int64_t n_pos,
         int32_t n_freq, int32_t interleaved, int32_t inverse, int32_t in_dtype,
         int32_t out_dtype, void *stream)
{
    if (!x || !y || !positions || !table)
        return BQM_ERR_NULL;
    if (T < 0 || T > (1 << 23) || n_heads < 1 || head_dim < 2 || head_dim > 1024 ||
        (int64_t)n_heads * head_dim > (1 << 23) || n_freq < 1 || 2 * (int64_t)n_freq > head_dim ||
        n_pos < 1 || n_pos > 0x7fffffff || !is_dtype(in_dtype) || !is_dtype(out_dtype))
        return BQM_ERR_SHAPE;
    for (const int64_t s : {x_token_stride, x_head_stride, y_token_stride, y_head_stride})
        if (s < 0 || s > (1ll << 38))
            return BQM_ERR_SHAPE;
    // in place every value is read and written by one thread: same places only
    if (x == y && (in_dtype != out_dtype || x_token_stride != y_token_stride ||
                   x_head_stride != y_head_stride))
        return BQM_ERR_SHAPE;
    if (!aligned(x, bytes_of(in_dtype)) || !aligned(y, bytes_of(out_dtype)) ||
        !aligned4(positions) || !aligned(table, 8))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    if (T == 0)
        return BQM_OK;
    return bqm::launch_rope(x, x_token_stride, x_head_stride, y, y_token_stride, y_head_stride,
                            positions, table, T, n_heads, head_dim, n_pos, n_freq,
                            interleaved != 0, inverse != 0, in_dtype, out_dtype,
                            as_stream(stream));
}

int rope_kv_append(const void *q, const void *k, const void *v, int64_t token_stride, void *q_out,
                   const bqm_kv_cache *cache, const bqm_kv_batch *batch, const int32_t *positions,
                   const float *table, int64_t n_pos, int32_t n_freq, int32_t interleaved,
                   int32_t n_q_heads, int32_t in_dtype, void *stream)
{
    if (!k || !v || !table || n_q_heads < 0 || (n_q_heads > 0 && (!q || !q_out)))
        return n_q_heads < 0 ? BQM_ERR_SHAPE : BQM_ERR_NULL;
    if (int rc = check_cache(cache))
        return rc;
    if (int rc = check_batch(batch))
        return rc;
    if (((int64_t)n_q_heads + 2 * (int64_t)cache->n_heads) * cache->head_dim > (1 << 23) ||
        n_freq < 1 || 2 * (int64_t)n_freq > cache->head_dim || n_pos < 1 || n_pos > 0x7fffffff ||
        token_stride < 0 || token_stride > (1ll << 38) || !is_dtype(in_dtype))
        return BQM_ERR_SHAPE;
    const uintptr_t e = bytes_of(in_dtype);
    if (!aligned(k, e) || !aligned(v, e) || (n_q_heads > 0 && (!aligned(q, e) || !aligned(q_out, 16))) ||
        !aligned(table, 8) || (positions && !aligned4(positions)))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    if (batch->total_q == 0)
        return BQM_OK;
    return bqm::launch_rope_append(n_q_heads > 0 ? q : nullptr, k, v, token_stride, q_out, cache,
                                   batch, positions, table, n_pos, n_freq, interleaved != 0,
                                   n_q_heads, in_dtype, as_stream(stream));
}

static bool attention_heads_ok(const bqm_kv_cache *c, const bqm_kv_batch *b, int32_t n_q_heads)
{
    return b->total_q * n_q_heads <= 0x7fffffff &&
           n_q_heads >= 1 && n_q_heads <= 65535 && n_q_heads % c->n_heads == 0 &&
           (int64_t)n_q_heads * c->head_dim <= (1 << 23);
}

size_t paged_attention_workspace_bytes(const bqm_kv_cache *cache, const bqm_kv_batch *batch,
                                       int32_t n_q_heads)
{
    if (check_cache(cache) || !batch || batch->n_seqs < 1 || batch->n_seqs > 65535 ||
        batch->max_pages < 1 || batch->total_q < 0 || batch->total_q > (1 << 23) ||
        batch->max_q < 0 || batch->max_kv < 0 || batch->max_kv > (1 << 30) ||
        !attention_heads_ok(cache, batch, n_q_heads))
        return 0;
    return bqm::attention_workspace(cache, batch, n_q_heads);
}

int paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                    const bqm_kv_cache *cache, const bqm_kv_batch *batch, void *out,
                    int32_t n_q_heads, float scale, int32_t causal, int32_t window,
                    int32_t out_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!q || !out)
        return BQM_ERR_NULL;
    if (int rc = check_cache(cache))
        return rc;
    if (int rc = check_batch(batch))
        return rc;
    if (!attention_heads_ok(cache, batch, n_q_heads) || !(scale > 0.0f) || !isfinite(scale) ||
        window < 0 || (out_dtype != cache->dtype && out_dtype != BQM_DTYPE_F32) ||
        q_token_stride < 0 || q_token_stride > (1ll << 38) || q_head_stride < 0 ||
        q_head_stride > (1ll << 38))
        return BQM_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || (q_token_stride | q_head_stride) % 8 != 0)
        return BQM_ERR_ALIGN;
    const size_t need = bqm::attention_workspace(cache, batch, n_q_heads);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return BQM_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    if (batch->total_q == 0)
        return BQM_OK;
    return bqm::launch_paged_attention(q, q_token_stride, q_head_stride, cache, batch, out,
                                       n_q_heads, scale, causal != 0, window, out_dtype, workspace,
                                       as_stream(stream));
}

static int check_pages(const bqm_kv_pages *p)
{
    if (!p || !p->table || !p->lens || !p->refs)
        return BQM_ERR_NULL;
    if (p->n_pages < 1 || p->n_pages > (1 << 30) || p->n_seqs < 1 || p->n_seqs > 65535 ||
        p->max_pages < 1 || p->max_pages > (1 << 24) || p->table_stride < p->max_pages)
        return BQM_ERR_SHAPE;
    if (!aligned4(p->table) || !aligned4(p->lens) || !aligned4(p->refs))
        return BQM_ERR_ALIGN;
    return BQM_OK;
}

static int check_in_out(const bqm_kv_pages *in, const bqm_kv_pages *out)
{
    if (int rc = check_pages(in))
        return rc;
    if (int rc = check_pages(out))
        return rc;
    if (in->n_pages != out->n_pages || in->n_seqs != out->n_seqs ||
        in->max_pages != out->max_pages ||
        (in->table == out->table && in->table_stride != out->table_stride))
        return BQM_ERR_SHAPE;
    return BQM_OK;
}

static int check_pages_workspace(const bqm_kv_pages *p, const void *workspace, size_t bytes)
{
    if (!workspace || bytes < bqm::kv_pages_workspace(p->n_pages, p->n_seqs))
        return BQM_ERR_WORKSPACE;
    return aligned(workspace, 256) ? BQM_OK : BQM_ERR_ALIGN;
}

static bool page_size_ok(int32_t n) { return n >= 1 && n <= 65536; }

size_t kv_pages_workspace_bytes(const bqm_kv_pages *pages)
{
    if (!pages || pages->n_pages < 1 || pages->n_pages > (1 << 30) || pages->n_seqs < 1 ||
        pages->n_seqs > 65535)
        return 0;
    return bqm::kv_pages_workspace(pages->n_pages, pages->n_seqs);
}

int kv_extend(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *n_new,
              int32_t page_size, int32_t *short_of, void *workspace, size_t workspace_bytes,
              void *stream)
{
    if (!n_new || !short_of)
        return BQM_ERR_NULL;
    if (int rc = check_in_out(in, out))
        return rc;
    if (!page_size_ok(page_size))
        return BQM_ERR_SHAPE;
    if (!aligned4(n_new) || !aligned4(short_of))
        return BQM_ERR_ALIGN;
    if (int rc = check_pages_workspace(in, workspace, workspace_bytes))
        return rc;
    if (int rc = check_device())
        return rc;
    return bqm::launch_kv_extend(in, out, n_new, page_size, short_of, workspace,
                                 as_stream(stream));
}

int kv_fork(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *parents,
            const int32_t *children, int32_t n, int32_t page_size, int32_t *moves,
            int32_t *short_of, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!parents || !children || !moves || !short_of)
        return BQM_ERR_NULL;
    if (int rc = check_in_out(in, out))
        return rc;
    if (!page_size_ok(page_size) || n < 0 || n > in->n_seqs)
        return BQM_ERR_SHAPE;
    if (!aligned4(parents) || !aligned4(children) || !aligned4(moves) || !aligned4(short_of))
        return BQM_ERR_ALIGN;
    if (int rc = check_pages_workspace(in, workspace, workspace_bytes))
        return rc;
    if (int rc = check_device())
        return rc;
    return bqm::launch_kv_fork(in, out, parents, children, n, page_size, moves, short_of,
                               workspace, as_stream(stream));
}

int kv_free(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *seqs, int32_t n,
            void *stream)
{
    if (!seqs)
        return BQM_ERR_NULL;
    if (int rc = check_in_out(in, out))
        return rc;
    if (n < 0 || n > 65535)
        return BQM_ERR_SHAPE;
    if (!aligned4(seqs))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_kv_free(in, out, seqs, n, as_stream(stream));
}

int kv_compact(const bqm_kv_pages *in, const bqm_kv_pages *out, int32_t page_size,
               int32_t *page_map, int32_t *moves, void *stream)
{
    if (!page_map || !moves)
        return BQM_ERR_NULL;
    if (int rc = check_in_out(in, out))
        return rc;
    if (!page_size_ok(page_size))
        return BQM_ERR_SHAPE;
    if (!aligned4(page_map) || !aligned4(moves))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return bqm::launch_kv_compact(in, out, page_size, page_map, moves, as_stream(stream));
}

int kv_copy_pages(const bqm_kv_cache *cache, const int32_t *moves, int64_t n, void *stream)
{
    if (!moves)
        return BQM_ERR_NULL;
    if (int rc = check_cache(cache))
        return rc;
    if (n < 0 || n > (1 << 30))
        return BQM_ERR_SHAPE;
    if (!aligned4(moves))
        return BQM_ERR_ALIGN;
    if (int rc = check_device())
        return rc;
    return n == 0 ? BQM_OK : bqm::launch_kv_copy_pages(cache, moves, n, as_stream(stream));
}

const char *bqm_status_string(int status)
{
    switch (status) {
    case BQM_OK:
        return "ok";
    case BQM_ERR_NULL:
        return "a required pointer is NULL";
    case BQM_ERR_SHAPE:
        return "a size is out of range";
    case BQM_ERR_ALIGN:
        return "a buffer is misaligned";
    case BQM_ERR_WORKSPACE:
        return "workspace missing or too small";
    case BQM_ERR_LAUNCH:
        return "the HIP runtime reported a launch error";
    case BQM_ERR_DEVICE:
        return "the current device is not a gfx950 GPU";
    default:
        return "unknown status";
    }
}

int bqm_version(void) { return kVersion; }

}  // extern "C"
