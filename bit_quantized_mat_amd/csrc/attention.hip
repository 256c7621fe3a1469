// attention.hip -- attention of new tokens over a paged cache.
//
// out = sum_j e_j v_j / sum_j e_j, e_j = exp(scale q.k_j - max): one pass over
// the keys with the running maximum and sum.
#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

struct AttnArgs {
    const void *q, *k, *v;
    void *out;
    const int32_t *pages, *kv_lens, *q_starts;
    int64_t q_token, q_head, pages_stride;
    int64_t c_page, c_token, c_head;
    int64_t total_q, n_pages;
    int n_seqs, max_pages, page_size, max_q, max_kv;
    int n_q_heads, group, dim;
    float scale;
    int causal, window;
};

// One wave per query head and token: each lane scores one key of 64, then the
// lanes hold the output's values and the keys go by one at a time.
template <class T, class O>
__global__ __launch_bounds__(64) void attention_plain_kernel(AttnArgs a)
{
    __shared__ float qs[256];
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, lane = threadIdx.x;
    int lo = 0, hi = a.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.q_starts[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const T *q = static_cast<const T *>(a.q) + t * a.q_token + h * a.q_head;
    for (int d = lane; d < a.dim; d += 64)
        qs[d] = (float)q[d];
    __syncthreads();
    const int most = (int)min((int64_t)a.max_kv, (int64_t)a.max_pages * a.page_size);
    const int kv_len = min(a.kv_lens[lo], most);
    const int pos = (int)(kv_len - a.q_starts[lo + 1] + t);
    int first = 0, end = kv_len;
    if (a.causal)
        end = min(end, pos + 1);
    if (a.window > 0)
        first = (int)max((int64_t)0, (int64_t)pos - a.window + 1);
    const T *kc = static_cast<const T *>(a.k) + h / a.group * a.c_head;
    const T *vc = static_cast<const T *>(a.v) + h / a.group * a.c_head;
    float top = -INFINITY, sum = 0.0f, acc[4] = {};
    for (int j0 = first; j0 < end; j0 += 64) {
        const int j = j0 + lane;
        float s = -INFINITY;
        int64_t at = -1;
        if (j < end) {
            const int page = a.pages[lo * a.pages_stride + j / a.page_size];
            s = 0.0f;
            if ((uint64_t)(int64_t)page < (uint64_t)a.n_pages) {
                at = page * a.c_page + (j % a.page_size) * a.c_token;
                for (int d = 0; d < a.dim; d++)
                    s += qs[d] * (float)kc[at + d];
            }
            s *= a.scale;
        }
        float m = s;
        for (int x = 32; x >= 1; x >>= 1)
            m = fmaxf(m, __shfl_xor(m, x, 64));
        m = fmaxf(m, top);
        const float back = expf(top - m);
        const float p = (float)(T)expf(s - m);
        float add = j < end ? p : 0.0f;
        for (int x = 32; x >= 1; x >>= 1)
            add += __shfl_xor(add, x, 64);
        sum = sum * back + add;
        top = m;
        for (int c = 0; c < 4; c++)
            acc[c] *= back;
        for (int e = 0; e < 64 && j0 + e < end; e++) {
            const float pe = __shfl(p, e, 64);
            const int64_t ae = __shfl(at, e, 64);
            if (ae >= 0)
                for (int c = 0; c < 4; c++)
                    if (c * 64 + lane < a.dim)
                        acc[c] += pe * (float)vc[ae + c * 64 + lane];
        }
    }
    O *out = static_cast<O *>(a.out) + (t * a.n_q_heads + h) * (int64_t)a.dim;
    for (int c = 0; c < 4; c++)
        if (c * 64 + lane < a.dim)
            out[c * 64 + lane] = (O)(sum == 0.0f ? 0.0f : acc[c] / sum);
}

}  // namespace

size_t attention_workspace(const bqm_kv_cache *, const bqm_kv_batch *, int) { return 0; }

int launch_paged_attention(const void *q, int64_t q_token, int64_t q_head, const bqm_kv_cache *c,
                           const bqm_kv_batch *b, void *out, int n_q_heads, float scale,
                           bool causal, int window, int out_dtype, void *, hipStream_t stream)
{
    const AttnArgs a = {q, c->k, c->v, out, b->table, b->kv_lens, b->q_starts, q_token, q_head,
                        b->table_stride, c->page_stride, c->token_stride, c->head_stride,
                        b->total_q, c->n_pages, b->n_seqs, b->max_pages, c->page_size, b->max_q,
                        b->max_kv, n_q_heads, n_q_heads / c->n_heads, c->head_dim, scale, causal,
                        window};
    const dim3 grid((unsigned)b->total_q, (unsigned)n_q_heads);
    if (c->dtype == BQM_DTYPE_F16 && out_dtype == BQM_DTYPE_F32)
        hipLaunchKernelGGL((attention_plain_kernel<_Float16, float>), grid, dim3(64), 0, stream, a);
    else if (c->dtype == BQM_DTYPE_F16)
        hipLaunchKernelGGL((attention_plain_kernel<_Float16, _Float16>), grid, dim3(64), 0, stream, a);
    else if (out_dtype == BQM_DTYPE_F32)
        hipLaunchKernelGGL((attention_plain_kernel<__bf16, float>), grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL((attention_plain_kernel<__bf16, __bf16>), grid, dim3(64), 0, stream, a);
    return check_launch();
}

}  // namespace bqm
