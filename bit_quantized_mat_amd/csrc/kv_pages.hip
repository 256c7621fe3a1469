// kv_pages.hip -- upkeep of a paged key/value cache: which sequence holds
// which pages (extend, fork, free, compact), and the copies between pages
// that a fork or a compaction asks for.
//
// The bookkeeping is ranks: request r of a call (counted in the requests' order)
// takes the r-th lowest free page, so the result is a function of the inputs alone.
// Ranks are two exclusive scans, over the requests and over the free pages; one
// workgroup of 16 waves does both at once (6.3 us for 4 forks, one after the other
// 7.1), and a second launch of one wave per row rewrites the table. Tables of at most
// kOneLaunch entries take one launch for both. Latency bounds these launches (scans and
// loads that follow each other): 2 to 6 us for 8 sequences, 6.6 us and 4.6 us for 480
// sequences over 3115 pages.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWaves = kPlanThreads / 64;
constexpr int kRowThreads = 256;

// Counts are 32 bits wide and stop at kMany, above every rank that is given.
constexpr uint32_t kMany = (1u << 30) + 1;

__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) { return min(a + b, kMany); }

// Exclusive scans over the plan workgroup's threads, N at once (values at most kMany);
// total is everybody's.
template <int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (&total)[N])
{
    __shared__ uint32_t sums[N][kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t upto[N], before[N];
#pragma unroll
    for (int k = 0; k < N; k++)
        upto[k] = v[k];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int k = 0; k < N; k++) {
            const uint32_t u = __shfl_up(upto[k], d, 64);
            upto[k] = lane >= d ? add_up(upto[k], u) : upto[k];
        }
#pragma unroll
    for (int k = 0; k < N; k++) {
        before[k] = __shfl_up(upto[k], 1, 64);
        before[k] = lane == 0 ? 0 : before[k];
    }
    __syncthreads();  // the last call's readers are done
    if (lane == 63)
#pragma unroll
        for (int k = 0; k < N; k++)
            sums[k][wave] = upto[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) {
        uint32_t all = 0, waves_before = 0;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            waves_before = w == wave ? all : waves_before;
            all = add_up(all, sums[k][w]);
        }
        total[k] = all;
        v[k] = add_up(waves_before, before[k]);
    }
}

// The threads' greatest v, and the sum of their counts n (at most kMany).
__device__ __forceinline__ void block_max_and_sum(uint32_t &v, uint32_t &n)
{
    __shared__ uint32_t tops[kWaves], sums[kWaves];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        v = max(v, (uint32_t)__shfl_xor(v, d, 64));
        n = add_up(n, (uint32_t)__shfl_xor(n, d, 64));
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = v;
        sums[threadIdx.x >> 6] = n;
    }
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        v = max(v, tops[w]);
        n = add_up(n, sums[w]);
    }
}

struct Pages {
    const int32_t *table, *lens, *refs;
    int32_t *table_out, *lens_out, *refs_out;
    int64_t stride, stride_out;
    int n_pages, n_seqs, max_pages, page_size;
};

// Which pages are in use, 64 to a word, with the count of used pages before each
// word: a page's rank among the used (or free) ones is then a popcount. Words of
// kSegment pages at a time lie in LDS (tables beyond that are gone through again
// segment by segment).
constexpr int kWords = 4096;
constexpr int64_t kSegment = 64 * kWords;

class UsedPages {
  public:
    // All threads. Sends out the first loads of count(), for what the caller reads
    // meanwhile.
    __device__ void start(const Pages &p) { read(p, 0, threadIdx.x >> 6, ahead_); }

    // All threads, after start(). Counts the pages in use; beside that scan, the
    // caller's: before is the sum of the threads' before this one, total of all.
    __device__ int64_t count(const Pages &p, uint32_t mine = 0, uint32_t *before = nullptr,
                             uint32_t *total = nullptr)
    {
        uint32_t v[2] = {0, mine}, all[2];
        int64_t used = load(p, 0, 0, v, all, true);
        if (before) {
            *before = v[1];
            *total = all[1];
        }
        for (int64_t at = kSegment; at < p.n_pages; at += kSegment)
            used = load(p, at, used);
        return used;
    }

    // All threads, after count(): used pages before `page`, which exists.
    __device__ int64_t before(const Pages &p, int64_t page)
    {
        int64_t used = 0, at = 0;
        if (p.n_pages > kSegment) {
            for (; at + kSegment <= page; at += kSegment)
                used = load(p, at, used);
            load(p, at, used);
        }
        const int i = (int)(page - at);
        return (int64_t)before_()[i >> 6] +
               __popcll(masks_()[i >> 6] & ((1ull << (i & 63)) - 1));
    }

    // All threads, after count(): f(page, its count, used pages before it) of every
    // page, neighbouring threads on neighbouring pages.
    template <class F>
    __device__ void each(const Pages &p, F f)
    {
        int64_t used = 0;
        for (int64_t at = 0; at < p.n_pages; at += kSegment) {
            if (p.n_pages > kSegment)
                used = load(p, at, used);
            const int n = (int)min(kSegment, p.n_pages - at);
#pragma unroll 4
            for (int i = threadIdx.x; i < n; i += kPlanThreads) {
                const uint64_t lower = masks_()[i >> 6] & ((1ull << (i & 63)) - 1);
                f(at + i, p.refs[at + i], (int64_t)before_()[i >> 6] + __popcll(lower));
            }
        }
    }

  private:
    __device__ static uint64_t *masks_()
    {
        __shared__ uint64_t masks[kWords];
        return masks;
    }
    __device__ static int *before_()
    {
        __shared__ int before[kWords];
        return before;
    }

    static constexpr int kAhead = 4;  // loads in flight of a thread
    int ahead_[kAhead];

    // Counts of word w's pages and of those a workgroup's stride of words apart
    __device__ static void read(const Pages &p, int64_t at, int w, int (&r)[kAhead])
    {
        const int n = (int)min(kSegment, p.n_pages - at);
#pragma unroll
        for (int k = 0; k < kAhead; k++)
            r[k] = p.refs[at + min((w + k * kWaves) * 64 + (int)(threadIdx.x & 63), n - 1)];
    }

    __device__ int64_t load(const Pages &p, int64_t at, int64_t used)
    {
        uint32_t v[1] = {0}, all[1];
        return load(p, at, used, v, all, false);
    }

    // The segment from page `at` on, `used` pages being in use before it; returns
    // the count after it. v, total: block_scan's, the first place for this one's use.
    template <int N>
    __device__ int64_t load(const Pages &p, int64_t at, int64_t used, uint32_t (&v)[N],
                            uint32_t (&total)[N], bool started)
    {
        const int n = (int)min(kSegment, p.n_pages - at), words = (n + 63) / 64;
        __syncthreads();  // the last segment's readers are done
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        for (int w0 = wave; w0 < words; w0 += kWaves * kAhead) {
            int r[kAhead];
            if (started && w0 == wave)
#pragma unroll
                for (int k = 0; k < kAhead; k++)
                    r[k] = ahead_[k];
            else
                read(p, at, w0, r);
#pragma unroll
            for (int k = 0; k < kAhead; k++) {
                const int w = w0 + k * kWaves;
                const uint64_t m = __ballot(w * 64 + lane < n && r[k] > 0);
                if (lane == 0 && w < words)
                    masks_()[w] = m;
            }
        }
        __syncthreads();
        constexpr int kPer = kWords / kPlanThreads;
        v[0] = 0;
        for (int w = threadIdx.x * kPer; w < min(words, (int)(threadIdx.x + 1) * kPer); w++)
            v[0] += __popcll(masks_()[w]);
        block_scan(v, total);
        int64_t first = used + v[0];
        for (int w = threadIdx.x * kPer; w < min(words, (int)(threadIdx.x + 1) * kPer); w++) {
            before_()[w] = (int)first;
            first += __popcll(masks_()[w]);
        }
        __syncthreads();
        return used + total[0];
    }
};

// This thread's run of n items, in the threads' order.
__device__ __forceinline__ void run_of(int64_t n, int64_t *lo, int64_t *hi)
{
    const int64_t per = (n + kPlanThreads - 1) / kPlanThreads;
    *lo = threadIdx.x * per < n ? threadIdx.x * per : n;
    *hi = *lo + per < n ? *lo + per : n;
}

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
    int32_t *tokens;     // [n] of each fork's parent, before any row is written: a parent
                         // may itself be a child, whose length in place changes meanwhile
    int n;
};

struct Wish {
    int have, need;  // pages
    bool fits;       // the row holds the grown sequence
};

// Pages of n tokens, n below 2^32.
__device__ __forceinline__ uint32_t pages_for(uint32_t n, int page_size)
{
    return n == 0 ? 0u : (n - 1) / (uint32_t)page_size + 1;
}

__device__ __forceinline__ Wish wish_of(const Pages &p, const Extend &e, int64_t s)
{
    const uint32_t len = max(p.lens[s], 0), grown = len + (uint32_t)max(e.n_new[s], 0);
    Wish w;
    w.have = (int)pages_for(len, p.page_size);
    const uint32_t want = pages_for(grown, p.page_size);
    w.fits = grown == len || (want <= (uint32_t)p.max_pages && grown <= 0x7fffffffu);
    w.need = w.fits ? (int)want - w.have : 0;
    return w;
}

// Gives the free pages of rank below `granted` (each is then held once) and
// lists them.
__device__ __forceinline__ void give_pages(const Pages &p, UsedPages &u, int32_t *free_list,
                                           int64_t granted)
{
    u.each(p, [&](int64_t i, int r, int64_t used_before) {
        const int64_t rank = i - used_before;
        if (r <= 0 && rank < granted) {
            free_list[rank] = (int)i;
            r = 1;
        }
        p.refs_out[i] = r;
    });
}

__device__ void extend_plan(const Pages &p, const Extend &e)
{
    UsedPages pages;
    int64_t lo, hi;
    uint32_t rank, total, mine = 0;
    pages.start(p);
    run_of(p.n_seqs, &lo, &hi);
    for (int64_t s = lo; s < hi; s++)
        mine = add_up(mine, wish_of(p, e, s).need);
    const uint32_t n_free = (uint32_t)(p.n_pages - pages.count(p, mine, &rank, &total));
    uint32_t granted = 0, refused = 0;
    for (int64_t s = lo; s < hi; s++) {
        const Wish w = wish_of(p, e, s);
        const uint32_t end = add_up(rank, w.need);
        const bool served = w.fits && (w.need == 0 || end <= n_free);
        refused += !served;
        if (served && w.need > 0)
            granted = end;
        e.first[s] = served && w.need > 0 ? (int)rank : -1;
        e.have[s] = w.have;
        e.need[s] = w.need;
        p.lens_out[s] = served ? max(p.lens[s], 0) + max(e.n_new[s], 0) : p.lens[s];
        rank = end;
    }
    block_max_and_sum(granted, refused);
    if (threadIdx.x == 0)
        e.short_of[0] = (int)refused;
    give_pages(p, pages, e.free_list, granted);
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
    UsedPages pages;
    int64_t lo, hi;
    uint32_t rank, total, mine = 0;
    pages.start(p);
    run_of(f.n, &lo, &hi);
    for (int64_t i = lo; i < hi; i++) {
        const int len = fork_length(p, f, i);
        mine += len > 0 && len % p.page_size != 0;
    }
    const uint32_t n_free = (uint32_t)(p.n_pages - pages.count(p, mine, &rank, &total));
    give_pages(p, pages, f.free_list, min(total, n_free));
    for (int64_t s = threadIdx.x; s < p.n_seqs; s += kPlanThreads)
        f.fork_of[s] = -1;
    __syncthreads();
    for (int64_t i = lo; i < hi; i++) {
        const int len = fork_length(p, f, i);
        int from = -1, to = -1, tail = 0;
        if (len >= 0) {
            tail = len % p.page_size;
            if (tail > 0) {
                if (rank < n_free) {
                    from = p.table[f.parents[i] * p.stride + len / p.page_size];
                    to = f.free_list[rank];
                }
                rank++;
            }
            f.fork_of[f.children[i]] = (int)i;
        }
        f.tokens[i] = len;
        f.moves[3 * i] = from;
        f.moves[3 * i + 1] = to;
        f.moves[3 * i + 2] = to < 0 ? 0 : tail;
    }
    if (threadIdx.x == 0)
        f.short_of[0] = (int)(total - min(total, n_free));
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
    int len = f.tokens[i];
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
    UsedPages pages;
    pages.start(p);
    const int64_t used = pages.count(p);
    // used pages below the cut; the rest of them move
    const int64_t low_used = used < p.n_pages ? pages.before(p, used) : used;
    const int64_t n = used - low_used;
    pages.each(p, [&](int64_t i, int r, int64_t u) {
        if (r > 0) {
            if (i >= used)
                moves[3 * (u - low_used)] = (int)i;
        } else if (i < used) {
            moves[3 * (i - u) + 1] = (int)i;  // i - u free pages lie before i
        }
        page_map[i] = (int)i;
        p.refs_out[i] = r;
    });
    __syncthreads();
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
constexpr int kCopyUnroll = 4;

struct CopyArgs {
    u32x4 *k, *v;                           // a 16-byte piece is 8 values
    int64_t layer, page, token, head;       // strides in pieces
    const int32_t *moves;
    int64_t n_pages;
    int page_size, n_heads, pieces;         // pieces of one head
};

// Memory bounds the copies. Reads and writes pass the caches by (nothing is read
// twice): moves of 1.7 GB, read and written, 315 us (5.4 TB/s) where cached ones took
// 458; four pieces a thread in flight, eight 8 us slower.
//
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
    u32x4 *base = (blockIdx.y & 1 ? a.v : a.k) + (int64_t)(blockIdx.y >> 1) * a.layer;
    const u32x4 *src = base + from * a.page;
    u32x4 *dst = base + to * a.page;
    const int row = a.n_heads * a.pieces;
    const int64_t all = (int64_t)tokens * row;
    const int64_t step = (int64_t)shares * kCopyThreads;
    for (int64_t i0 = (int64_t)share * kCopyThreads + threadIdx.x; i0 < all;
         i0 += step * kCopyUnroll) {
        u32x4 x[kCopyUnroll];
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
                x[u] = __builtin_nontemporal_load(src + at[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; u++)
            if (at[u] >= 0)
                __builtin_nontemporal_store(x[u], dst + at[u]);
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
    int32_t *per_seq = ws + p.n_pages;
    const Fork f = {parents, children, moves, short_of, ws, per_seq, per_seq + p.n_seqs, n};
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
    const CopyArgs a = {static_cast<u32x4 *>(c->k), static_cast<u32x4 *>(c->v),
                        c->layer_stride / 8, c->page_stride / 8, c->token_stride / 8,
                        c->head_stride / 8, moves, c->n_pages,
                        c->page_size, c->n_heads, c->head_dim / 8};
    const bool flat = (c->n_heads == 1 || c->head_stride == c->head_dim) &&
                      (c->page_size == 1 || c->token_stride == (int64_t)c->n_heads * c->head_dim);
    // a share of a page is at least 16 KiB (4 pieces a thread)
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
