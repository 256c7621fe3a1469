// kv_pages.hip -- upkeep of a paged key/value cache: which sequence holds
// which pages (extend, fork, free, compact), and the copies between pages
// that a fork or a compaction asks for.
//
// The bookkeeping is ranks: request r of a call (counted in the requests'
// order) takes the r-th lowest free page, so the result is a function of the
// inputs alone. Ranks are two exclusive scans, over the requests and over the
// free pages; one workgroup of 16 waves does both (a table of 100000 pages is
// 400 KB, which one workgroup reads from L2 in the time of two launches), and
// a second launch of one wave per row rewrites the table. Tables of at most
// kOneLaunch entries take one launch for both.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWaves = kPlanThreads / 64;
constexpr int kRowThreads = 256;

__device__ __forceinline__ int64_t wave_inclusive_scan(int64_t v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t u = __shfl_up(v, d, 64);
        if (lane >= d)
            v += u;
    }
    return v;
}

// Exclusive scan over the plan workgroup's threads; *total is everybody's.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *total)
{
    __shared__ int64_t sums[kWaves];
    const int wave = threadIdx.x >> 6;
    const int64_t inc = wave_inclusive_scan(v);
    __syncthreads();  // the last call's readers are done
    if ((threadIdx.x & 63) == 63)
        sums[wave] = inc;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        before += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    *total = all;
    return before + inc - v;
}

__device__ __forceinline__ int64_t block_max(int64_t v)
{
    __shared__ int64_t tops[kWaves];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const int64_t u = __shfl_xor(v, d, 64);
        v = u > v ? u : v;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        tops[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < kWaves; w++)
        v = tops[w] > v ? tops[w] : v;
    return v;
}

// This thread's run of n items, in the threads' order.
__device__ __forceinline__ void run_of(int64_t n, int64_t *lo, int64_t *hi)
{
    const int64_t per = (n + kPlanThreads - 1) / kPlanThreads;
    *lo = threadIdx.x * per < n ? threadIdx.x * per : n;
    *hi = *lo + per < n ? *lo + per : n;
}

struct Pages {
    const int32_t *table, *lens, *refs;
    int32_t *table_out, *lens_out, *refs_out;
    int64_t stride, stride_out;
    int n_pages, n_seqs, max_pages, page_size;
};

struct Extend {
    const int32_t *n_new;
    int32_t *short_of;
    int32_t *free_list;  // workspace: [n_pages] page of each rank that is given
    int32_t *first;      // [n_seqs] rank of the row's first new page, -1: none
    int32_t *have;       // [n_seqs] pages before
    int32_t *need;       // [n_seqs] pages new
};

struct Fork {
    const int32_t *parents, *children;
    int32_t *moves, *short_of;
    int32_t *free_list;  // workspace, as above
    int32_t *fork_of;    // [n_seqs] the fork whose child the row is, -1: none
    int n;
};

struct Wish {
    int64_t have, need;
    bool fits;  // the row holds the grown sequence
};

__device__ __forceinline__ Wish wish_of(const Pages &p, const Extend &e, int64_t s)
{
    const int64_t len = max(p.lens[s], 0), grown = len + max(e.n_new[s], 0);
    Wish w;
    w.have = (len + p.page_size - 1) / p.page_size;
    const int64_t want = (grown + p.page_size - 1) / p.page_size;
    w.fits = grown == len || (want <= p.max_pages && grown <= 0x7fffffff);
    w.need = w.fits ? want - w.have : 0;
    return w;
}

// Gives the free pages of rank below `granted` (each to become held once) and
// lists them; returns nothing but what it wrote. base: this thread's first rank.
__device__ __forceinline__ void give_pages(const Pages &p, int32_t *free_list, int64_t base,
                                           int64_t granted)
{
    int64_t lo, hi;
    run_of(p.n_pages, &lo, &hi);
    for (int64_t i = lo; i < hi; i++) {
        int r = p.refs[i];
        if (r <= 0 && base < granted) {
            free_list[base] = (int)i;
            r = 1;
            base++;
        }
        p.refs_out[i] = r;
    }
}

__device__ __forceinline__ int64_t count_free(const Pages &p, int64_t *base)
{
    int64_t lo, hi, mine = 0, n_free;
    run_of(p.n_pages, &lo, &hi);
    for (int64_t i = lo; i < hi; i++)
        mine += p.refs[i] <= 0;
    *base = block_scan(mine, &n_free);
    return n_free;
}

__device__ void extend_plan(const Pages &p, const Extend &e)
{
    int64_t page_base, total, lo, hi, mine = 0;
    const int64_t n_free = count_free(p, &page_base);
    run_of(p.n_seqs, &lo, &hi);
    for (int64_t s = lo; s < hi; s++)
        mine += wish_of(p, e, s).need;
    int64_t rank = block_scan(mine, &total);
    int64_t granted = 0, refused = 0;
    for (int64_t s = lo; s < hi; s++) {
        const Wish w = wish_of(p, e, s);
        const int64_t end = rank + w.need;
        const bool served = w.fits && (w.need == 0 || end <= n_free);
        refused += !served;
        if (served && w.need > 0)
            granted = end;
        e.first[s] = served && w.need > 0 ? (int)rank : -1;
        e.have[s] = (int)w.have;
        e.need[s] = (int)w.need;
        p.lens_out[s] = served ? max(p.lens[s], 0) + max(e.n_new[s], 0) : p.lens[s];
        rank = end;
    }
    granted = block_max(granted);
    int64_t all;
    block_scan(refused, &all);
    if (threadIdx.x == 0)
        e.short_of[0] = (int)all;
    give_pages(p, e.free_list, page_base, granted);
}

// Row s of the table, by one wave.
__device__ void extend_row(const Pages &p, const Extend &e, int s)
{
    const int first = e.first[s], have = e.have[s], need = first < 0 ? 0 : e.need[s];
    for (int j = threadIdx.x & 63; j < p.max_pages; j += 64) {
        const int k = j - have;
        p.table_out[s * p.stride_out + j] =
            k >= 0 && k < need ? e.free_list[first + k] : p.table[s * p.stride + j];
    }
}

// Length of fork i's parent, or -1 for a fork that is left out.
__device__ __forceinline__ int fork_length(const Pages &p, const Fork &f, int64_t i)
{
    const int a = f.parents[i], c = f.children[i];
    if ((unsigned)a >= (unsigned)p.n_seqs || (unsigned)c >= (unsigned)p.n_seqs)
        return -1;
    const int64_t most = (int64_t)p.max_pages * p.page_size;
    return (int)min((int64_t)max(p.lens[a], 0), most);
}

__device__ void fork_plan(const Pages &p, const Fork &f)
{
    int64_t page_base, total, lo, hi, mine = 0;
    const int64_t n_free = count_free(p, &page_base);
    run_of(f.n, &lo, &hi);
    for (int64_t i = lo; i < hi; i++) {
        const int len = fork_length(p, f, i);
        mine += len > 0 && len % p.page_size != 0;
    }
    const int64_t rank0 = block_scan(mine, &total);
    give_pages(p, f.free_list, page_base, total < n_free ? total : n_free);
    for (int64_t s = threadIdx.x; s < p.n_seqs; s += kPlanThreads)
        f.fork_of[s] = -1;
    __syncthreads();
    int64_t rank = rank0, refused = 0;
    for (int64_t i = lo; i < hi; i++) {
        const int len = fork_length(p, f, i);
        int from = -1, to = -1, tail = 0;
        if (len >= 0) {
            tail = len % p.page_size;
            if (tail > 0) {
                if (rank < n_free) {
                    from = p.table[f.parents[i] * p.stride + len / p.page_size];
                    to = f.free_list[rank];
                } else {
                    refused++;
                }
                rank++;
            }
            f.fork_of[f.children[i]] = (int)i;
        }
        f.moves[3 * i] = from;
        f.moves[3 * i + 1] = to;
        f.moves[3 * i + 2] = to < 0 ? 0 : tail;
    }
    int64_t all;
    block_scan(refused, &all);
    if (threadIdx.x == 0)
        f.short_of[0] = (int)all;
}

__device__ void fork_row(const Pages &p, const Fork &f, int s)
{
    const int i = f.fork_of[s];
    if (i < 0) {
        if (p.table_out != p.table)
            for (int j = threadIdx.x & 63; j < p.max_pages; j += 64)
                p.table_out[s * p.stride_out + j] = p.table[s * p.stride + j];
        if ((threadIdx.x & 63) == 0)
            p.lens_out[s] = p.lens[s];
        return;
    }
    const int to = f.moves[3 * i + 1];
    int len = fork_length(p, f, i);
    if (len % p.page_size != 0 && to < 0)
        len = 0;  // no page was free
    const int full = len / p.page_size;
    const int32_t *row = p.table + f.parents[i] * p.stride;
    for (int j = threadIdx.x & 63; j < p.max_pages; j += 64) {
        int page = -1;
        if (j < full) {
            page = row[j];
            if ((unsigned)page < (unsigned)p.n_pages)
                atomicAdd(&p.refs_out[page], 1);  // whole numbers: any order
        } else if (j == full && len > 0) {
            page = to;
        }
        p.table_out[s * p.stride_out + j] = page;
    }
    if ((threadIdx.x & 63) == 0)
        p.lens_out[s] = len;
}

__device__ void free_row(const Pages &p, const int32_t *seqs, int n, int s)
{
    const int lane = threadIdx.x & 63;
    bool listed = false;
    for (int i = lane; i < n; i += 64)
        listed |= seqs[i] == s;
    listed = __any(listed);
    for (int j = lane; j < p.max_pages; j += 64) {
        const int page = p.table[s * p.stride + j];
        if (listed && (unsigned)page < (unsigned)p.n_pages)
            atomicSub(&p.refs_out[page], 1);
        p.table_out[s * p.stride_out + j] = listed ? -1 : page;
    }
    if (lane == 0)
        p.lens_out[s] = listed ? 0 : p.lens[s];
}

__device__ void copy_refs(const Pages &p, int64_t first, int64_t step)
{
    if (p.refs_out != p.refs)
        for (int64_t i = first; i < p.n_pages; i += step)
            p.refs_out[i] = p.refs[i];
}

__device__ void compact_plan(const Pages &p, int32_t *page_map, int32_t *moves)
{
    int64_t lo, hi, mine = 0, used;
    run_of(p.n_pages, &lo, &hi);
    for (int64_t i = lo; i < hi; i++)
        mine += p.refs[i] > 0;
    // used pages before this thread's run; free ones are the rest of them
    int64_t u = block_scan(mine, &used);
    int64_t used_before_cut = 0;  // of the pages below `used`
    for (int64_t i = lo; i < hi && i < used; i++)
        used_before_cut += p.refs[i] > 0;
    int64_t low_used;
    block_scan(used_before_cut, &low_used);
    for (int64_t i = lo; i < hi; i++) {
        const int r = p.refs[i];
        if (r > 0) {
            if (i >= used)
                moves[3 * (u - low_used)] = (int)i;
            u++;
        } else if (i < used) {
            moves[3 * (i - u) + 1] = (int)i;  // i - u free pages lie before i
        }
        page_map[i] = (int)i;
        p.refs_out[i] = r;
    }
    __syncthreads();
    const int64_t n = used - low_used;
    for (int64_t m = threadIdx.x; m < p.n_pages / 2; m += kPlanThreads) {
        if (m < n) {
            const int from = moves[3 * m], to = moves[3 * m + 1];
            moves[3 * m + 2] = p.page_size;
            page_map[from] = to;
            const int r = p.refs[from];  // in place: only this thread writes it
            p.refs_out[to] = r;
            p.refs_out[from] = 0;
        } else {
            moves[3 * m] = moves[3 * m + 1] = -1;
            moves[3 * m + 2] = 0;
        }
    }
}

__device__ void compact_row(const Pages &p, const int32_t *page_map, int s)
{
    for (int j = threadIdx.x & 63; j < p.max_pages; j += 64) {
        const int page = p.table[s * p.stride + j];
        p.table_out[s * p.stride_out + j] =
            (unsigned)page < (unsigned)p.n_pages ? page_map[page] : page;
    }
    if ((threadIdx.x & 63) == 0)
        p.lens_out[s] = p.lens[s];
}

// PLAN: this launch makes the plan (one workgroup); ROWS: it rewrites the rows.
template <bool PLAN, bool ROWS, class PlanOf, class RowOf>
__device__ __forceinline__ void upkeep(int n_seqs, PlanOf plan, RowOf row)
{
    if constexpr (PLAN)
        plan();
    if constexpr (PLAN && ROWS)
        __syncthreads();
    if constexpr (ROWS)
        for (int s = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6); s < n_seqs;
             s += gridDim.x * (blockDim.x >> 6))
            row(s);
}

template <bool PLAN, bool ROWS>
__global__ __launch_bounds__(kPlanThreads) void extend_kernel(Pages p, Extend e)
{
    upkeep<PLAN, ROWS>(
        p.n_seqs, [&] { extend_plan(p, e); }, [&](int s) { extend_row(p, e, s); });
}

template <bool PLAN, bool ROWS>
__global__ __launch_bounds__(kPlanThreads) void fork_kernel(Pages p, Fork f)
{
    upkeep<PLAN, ROWS>(
        p.n_seqs, [&] { fork_plan(p, f); }, [&](int s) { fork_row(p, f, s); });
}

template <bool PLAN, bool ROWS>
__global__ __launch_bounds__(kPlanThreads) void free_kernel(Pages p, const int32_t *seqs, int n)
{
    upkeep<PLAN, ROWS>(
        p.n_seqs,
        [&] {
            copy_refs(p, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
                      (int64_t)gridDim.x * blockDim.x);
        },
        [&](int s) { free_row(p, seqs, n, s); });
}

template <bool PLAN, bool ROWS>
__global__ __launch_bounds__(kPlanThreads) void compact_kernel(Pages p, int32_t *page_map,
                                                               int32_t *moves)
{
    upkeep<PLAN, ROWS>(
        p.n_seqs, [&] { compact_plan(p, page_map, moves); },
        [&](int s) { compact_row(p, page_map, s); });
}

// Table entries and pages up to which one launch does plan and rows.
constexpr int64_t kOneLaunch = 16384;

// both: one workgroup does plan and rows; else plan (a grid of plan_blocks
// workgroups; 0: none) and rows after each other.
template <class K, class... A>
int launch_upkeep(K both, K plan, K rows, int plan_blocks, const Pages &p, hipStream_t stream,
                  A... args)
{
    if (p.n_pages + (int64_t)p.n_seqs * p.max_pages <= kOneLaunch) {
        hipLaunchKernelGGL(both, dim3(1), dim3(kPlanThreads), 0, stream, p, args...);
        return check_launch();
    }
    if (plan_blocks > 0)
        hipLaunchKernelGGL(plan, dim3(plan_blocks), dim3(kPlanThreads), 0, stream, p, args...);
    const int per = kRowThreads / 64;
    hipLaunchKernelGGL(rows, dim3((p.n_seqs + per - 1) / per), dim3(kRowThreads), 0, stream, p,
                       args...);
    return check_launch();
}

Pages pages_of(const bqm_kv_pages *in, const bqm_kv_pages *out, int page_size)
{
    return {in->table,        in->lens,          in->refs,         out->table,
            out->lens,        out->refs,         in->table_stride, out->table_stride,
            (int)in->n_pages, (int)in->n_seqs,   (int)in->max_pages, page_size};
}

// ---- copies -----------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;

struct CopyArgs {
    uint4 *k, *v;                           // a 16-byte piece is 8 values
    int64_t layer, page, token, head;       // strides in pieces
    const int32_t *moves;
    int64_t n_pages;
    int page_size, n_heads, pieces;         // pieces of one head
};

// One workgroup: a share (blockIdx.x % shares) of one page of one layer of k
// or v. FLAT: tokens lie behind one another, a move is one run of bytes.
template <bool FLAT>
__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(CopyArgs a, int shares)
{
    const int64_t m = blockIdx.x / shares;
    const int share = blockIdx.x % shares;
    const int from = a.moves[3 * m], to = a.moves[3 * m + 1];
    const int tokens = min(a.moves[3 * m + 2], a.page_size);
    if (tokens <= 0 || (uint64_t)(int64_t)from >= (uint64_t)a.n_pages ||
        (uint64_t)(int64_t)to >= (uint64_t)a.n_pages || from == to)
        return;
    uint4 *base = (blockIdx.y & 1 ? a.v : a.k) + (int64_t)(blockIdx.y >> 1) * a.layer;
    const uint4 *src = base + from * a.page;
    uint4 *dst = base + to * a.page;
    const int row = a.n_heads * a.pieces;
    const int64_t all = (int64_t)tokens * row;
    const int64_t step = (int64_t)shares * kCopyThreads;
    for (int64_t i0 = (int64_t)share * kCopyThreads + threadIdx.x; i0 < all;
         i0 += step * kCopyUnroll) {
        uint4 x[kCopyUnroll];
        int64_t at[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; u++) {
            const int64_t i = i0 + u * step;
            at[u] = -1;
            if (i < all) {
                if constexpr (FLAT) {
                    at[u] = i;
                } else {
                    const int64_t t = i / row;
                    const int r = (int)(i - t * row), h = r / a.pieces;
                    at[u] = t * a.token + h * a.head + (r - h * a.pieces);
                }
                x[u] = src[at[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; u++)
            if (at[u] >= 0)
                dst[at[u]] = x[u];
    }
}

}  // namespace

size_t kv_pages_workspace(int64_t n_pages, int64_t n_seqs)
{
    return ((size_t)(n_pages + 3 * n_seqs) * 4 + 255) / 256 * 256;
}

int launch_kv_extend(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *n_new,
                     int page_size, int32_t *short_of, void *workspace, hipStream_t stream)
{
    const Pages p = pages_of(in, out, page_size);
    int32_t *ws = static_cast<int32_t *>(workspace);
    int32_t *per_seq = ws + p.n_pages;
    const Extend e = {n_new,   short_of,           ws,
                      per_seq, per_seq + p.n_seqs, per_seq + 2 * (int64_t)p.n_seqs};
    return launch_upkeep(extend_kernel<true, true>, extend_kernel<true, false>,
                         extend_kernel<false, true>, 1, p, stream, e);
}

int launch_kv_fork(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *parents,
                   const int32_t *children, int n, int page_size, int32_t *moves,
                   int32_t *short_of, void *workspace, hipStream_t stream)
{
    const Pages p = pages_of(in, out, page_size);
    int32_t *ws = static_cast<int32_t *>(workspace);
    const Fork f = {parents, children, moves, short_of, ws, ws + p.n_pages, n};
    return launch_upkeep(fork_kernel<true, true>, fork_kernel<true, false>,
                         fork_kernel<false, true>, 1, p, stream, f);
}

int launch_kv_free(const bqm_kv_pages *in, const bqm_kv_pages *out, const int32_t *seqs, int n,
                   hipStream_t stream)
{
    const Pages p = pages_of(in, out, 1);
    const int blocks =
        p.refs_out == p.refs ? 0 : (int)std::min<int64_t>((p.n_pages + 1023) / 1024, 256);
    return launch_upkeep(free_kernel<true, true>, free_kernel<true, false>,
                         free_kernel<false, true>, blocks, p, stream, seqs, n);
}

int launch_kv_compact(const bqm_kv_pages *in, const bqm_kv_pages *out, int page_size,
                      int32_t *page_map, int32_t *moves, hipStream_t stream)
{
    const Pages p = pages_of(in, out, page_size);
    return launch_upkeep(compact_kernel<true, true>, compact_kernel<true, false>,
                         compact_kernel<false, true>, 1, p, stream, page_map, moves);
}

int launch_kv_copy_pages(const bqm_kv_cache *c, const int32_t *moves, int64_t n,
                         hipStream_t stream)
{
    const CopyArgs a = {static_cast<uint4 *>(c->k), static_cast<uint4 *>(c->v),
                        c->layer_stride / 8, c->page_stride / 8, c->token_stride / 8,
                        c->head_stride / 8, moves, c->n_pages,
                        c->page_size, c->n_heads, c->head_dim / 8};
    const bool flat = (c->n_heads == 1 || c->head_stride == c->head_dim) &&
                      (c->page_size == 1 || c->token_stride == (int64_t)c->n_heads * c->head_dim);
    // a share of a page is at least 32 KiB (8 pieces a thread)
    const int64_t pieces = (int64_t)c->page_size * c->n_heads * a.pieces;
    const int shares =
        (int)std::clamp<int64_t>(pieces / (kCopyThreads * kCopyUnroll), 1, 64);
    // a grid holds 2^32 threads in x and 65535 workgroups in y: what is beyond
    // goes in further launches
    const int64_t most = (1 << 23) / shares;
    for (int64_t l = 0; l < c->n_layers; l += 16384)
        for (int64_t m = 0; m < n; m += most) {
            CopyArgs b = a;
            b.k += l * a.layer;
            b.v += l * a.layer;
            b.moves += 3 * m;
            const int64_t layers = std::min<int64_t>(16384, c->n_layers - l);
            hipLaunchKernelGGL(flat ? copy_pages_kernel<true> : copy_pages_kernel<false>,
                               dim3((unsigned)(std::min(most, n - m) * shares),
                                    (unsigned)(2 * layers)),
                               dim3(kCopyThreads), 0, stream, b, shares);
            if (int rc = check_launch())
                return rc;
        }
    return BQM_OK;
}

}  // namespace bqm
