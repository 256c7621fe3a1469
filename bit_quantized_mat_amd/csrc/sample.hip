// sample.hip -- the next token of each row of logits (definition in include/bqm.h).
//
// Every question the filters and the draw ask is of one kind: going down the sorted
// tokens, at which one does the running count reach k, or the running weight W? So
// nothing is sorted but the few tokens around an answer: one pass sums counts and
// weights of 2048 bins of equal width in logits (32 to a factor of 2 in weight, so
// bins are in the sorted order), sums over bins give the answer's bin, and the
// tokens of that bin (or of all bins up to it, where they are few) are gathered
// and sorted in LDS. Where one bin alone holds too many, its range of logits is cut
// again until few are left or all of them are equal, and equal ones are taken by
// their ids.
//
// Weights are whole numbers of 2^-44: sums are exact, atomics in any order give the
// same bits.
//
// A row is a workgroup's. Where rows are few and long, the two passes over all of a row
// (its largest logit; its bins) are shared by several workgroups each, launches of their
// own before it. What bounds it: of few rows the latency of a score of steps (one row of
// 32001 logits 21.6 us), else the fp64 weights and the passes over a row by one compute unit
// (256 rows of 100003 bf16 82 us: largest 9, bins 25, each gathering 6 to 9, the rest not taken
// apart; 64 of fp32, shared by 8: 7 + 14 us, then 32 of the row's own workgroup).
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;      // of a row's workgroup
constexpr int kPartThreads = 512;   // of a part's
constexpr int kBins = 2048;
constexpr int kPartsMax = 64;
constexpr int kFew = 2048;  // tokens that are sorted in LDS
constexpr int kSteps = 1024;  // of the table of powers, in a factor of 2
constexpr double kOne = 17592186044416.0;  // 2^44

// A row's part of the workspace: what its parts add up.
struct RowSums {
    u64 weight[kBins];
    uint32_t count[kBins];
    u64 kept;  // weights that min_p leaves
    u64 best[kPartsMax];
};

struct SampleArgs {
    const void *logits;
    int64_t row_stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *tokens;
    float *logprobs;
    RowSums *rows;  // where rows are shared
    int V, parts;
};

struct Lds {
    double power[kSteps];      // 2^(i / kSteps)
    u64 weight[kBins + 1];     // sums of the bins before each
    uint32_t count[kBins + 1];  // (or bounds of them, where top_k does not ask)
    u64 few[kFew];             // key << 32 | ~id, sorted downwards
    u64 upto[kFew];            // weights of those up to and with each
    u64 part[16];
    u64 found_w;               // an answer: the weights up to and with the token,
    uint32_t found_id;         // the token,
    int found_bin;
    uint32_t n, key_lo, key_hi;
};

struct PartLds {
    double power[kSteps];
    u64 weight[kBins];
    uint32_t count[kBins];
    u64 kept;
};

// f(i, value) for the logits from .. to - 1 of a row as they are, dealt to n threads, each
// one's in ascending order: 16 bytes at a time, kDeep of them on their way.
template <int kDeep, class V, class F>
__device__ __forceinline__ void each(const V *x, int from, int to, int n, F f)
{
    constexpr int kPer = 16 / sizeof(V);
    auto one = [&](int i, V v) { f(i, (float)v); };
    const int odd = (int)((16 - (reinterpret_cast<uintptr_t>(x + from) & 15)) & 15) / (int)sizeof(V);
    const int head = odd < to - from ? odd : to - from;
    const int tid = threadIdx.x;
    if (tid < head)
        one(from + tid, x[from + tid]);
    const int first = from + head, pieces = (to - first) / kPer;
    const u32x4 *p = reinterpret_cast<const u32x4 *>(x + first);
    auto piece = [&](int i, const u32x4 &raw) {
        V v[kPer];
        __builtin_memcpy(v, &raw, 16);
#pragma unroll
        for (int k = 0; k < kPer; k++)
            one(first + i * kPer + k, v[k]);
    };
    for (int i = tid; i < pieces; i += kDeep * n) {
        u32x4 raw[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; k++)
            raw[k] = p[i + k * n < pieces ? i + k * n : i];
#pragma unroll
        for (int k = 0; k < kDeep; k++)
            if (i + k * n < pieces)
                piece(i + k * n, raw[k]);
    }
    const int tail = first + pieces * kPer;
    if (tid < to - tail)
        one(tail + tid, x[tail + tid]);
}

// Ascending with the value.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ u64 largest(u64 a, u64 b) { return a > b ? a : b; }

// The largest of a thread's logits, the first of equal ones; NaN is none.
struct Top {
    float v = -__builtin_inff();
    int i = 0x7fffffff;

    __device__ __forceinline__ void see(int at, float u)
    {
        if (u > v) {
            v = u;
            i = at;
        }
    }
    __device__ __forceinline__ u64 packed() const
    {
        return (u64)key_of(v + 0.0f) << 32 | (uint32_t)~i;  // (-0 is 0)
    }
};

__device__ __forceinline__ u64 wave_largest(u64 v)
{
    for (int m = 32; m; m >>= 1)
        v = largest(v, __shfl_xor(v, m, 64));
    return v;
}

// A row's settings.
struct Settings {
    float heat, p, floor;
    int k;
    bool first;  // the first token is taken (written so that NaN settings do, too)

    __device__ __forceinline__ Settings(const SampleArgs &g, int t)
        : heat(g.temperature ? g.temperature[t] : 1.0f), p(g.top_p ? g.top_p[t] : 1.0f),
          floor(g.min_p ? g.min_p[t] : 0.0f), k(g.top_k ? g.top_k[t] : 0)
    {
        first = !(heat > 0.0f) || k == 1 || !(p > 0.0f) || !(floor <= 1.0f);
    }
};

__device__ __forceinline__ void fill_powers(double *power, int n)
{
    for (int i = threadIdx.x; i < kSteps; i += n)
        power[i] = exp2((double)i / kSteps);
}

// A logit's weight, a whole number of 2^-44, and bin.
struct Weights {
    const double *power;
    double top, c;  // the largest logit; kSteps * log2(e) / temperature
    bool infinite;

    __device__ __forceinline__ void set(const double *table, float largest_logit, float heat)
    {
        power = table;
        top = largest_logit;
        infinite = largest_logit == __builtin_inff();
        c = kSteps * 1.4426950408889634 / (double)heat;
    }

    // (of logits of which none is +infinity)
    __device__ __forceinline__ u64 of_finite(float v, int &bin) const
    {
        // what is further down, -infinity, NaN and what -infinity makes NaN round to nothing
        const double y = fmax(((double)v - top) * c, -46.0 * kSteps);
        const double f = floor(y);
        const int k = (int)f;
        bin = (-k) >> 5;
        // 2^(y / kSteps) = power of the whole part times e^r, r below 2^-10.5: the series'
        // third power leaves 2^-46, five roundings to fp32 of e^r - 1 at most 2^-32.2 (2^-33.0
        // is the most that 40 million values showed)
        const float r = (float)(y - f) * 6.7690154351557158e-4f;  // ln(2) / kSteps
        const float p = r * fmaf(r, fmaf(r, 0.16666667f, 0.5f), 1.0f);
        double w = power[k & (kSteps - 1)];
        w = __builtin_fma(w, (double)p, w);
        // in 2^52 .. 2^53 a double's last bit is 1: the sum rounds to a whole number
        w = ldexp(w, 44 + (k >> 10)) + 4503599627370496.0;
        return (u64)__double_as_longlong(w) & 0xfffffffffffffull;
    }

    __device__ __forceinline__ u64 of(float v, int &bin) const
    {
        if (!infinite)
            return of_finite(v, bin);
        bin = 0;
        return v == __builtin_inff() ? (u64)kOne : 0;
    }

    // No logit below this has a bin of at most `bin`; none above that, one of at least `bin`.
    __device__ __forceinline__ float least(int bin) const
    {
        if (infinite)
            return -__builtin_inff();
        const double v = top - (32.0 * (bin + 1) + 1.0) / c;
        return (float)(v - fabs(v) * 1e-6);
    }
    __device__ __forceinline__ float most(int bin) const
    {
        if (infinite || bin == 0)
            return __builtin_inff();
        const double v = top - (32.0 * bin - 2.0) / c;
        return (float)(v + fabs(v) * 1e-6);
    }
};

// Weights and, for top_k alone, counts of the bins of logits from .. to - 1, into LDS that
// holds zeros. (A count costs LDS as much as a weight.)
template <class V>
__device__ __forceinline__ u64 fill_bins(const V *x, int from, int to, int n, const Weights &w,
                                         u64 *weight, uint32_t *count, const Settings &set)
{
    const u64 least = (u64)ceil((double)set.floor * kOne);
    u64 kept = 0;
    auto fill = [&](auto weight_of, auto counts, auto floors) {
        each<2>(x, from, to, n, [&](int, float v) {
            int bin;
            const u64 u = weight_of(v, bin);
            if (u) {
                atomicAdd(&weight[bin], u);
                if constexpr (counts.value)
                    atomicAdd(&count[bin], 1u);
                if constexpr (floors.value)
                    kept += u >= least ? u : 0;
            }
        });
    };
    const std::true_type yes;
    const std::false_type no;
    auto any = [&](float v, int &bin) { return w.of(v, bin); };
    auto finite = [&](float v, int &bin) { return w.of_finite(v, bin); };
    if (w.infinite)
        fill(any, yes, yes);
    else if (set.k > 0)
        fill(finite, yes, yes);
    else if (set.floor > 0.0f)
        fill(finite, no, yes);
    else
        fill(finite, no, no);
    return set.floor > 0.0f ? kept : 0;
}

// How many tokens a bin of this weight holds at most: none weighs less than the bin's lower
// end, 2.2% below its upper one.
__device__ __forceinline__ uint32_t most_tokens(u64 weight, int bin, const double *power)
{
    const int k = -32 * (bin + 1);
    const double each = ldexp(power[k & (kSteps - 1)], 44 + (k >> 10)) * 0.9999 - 0.5;
    return weight ? (uint32_t)((double)weight / (each > 1.0 ? each : 1.0)) + 1 : 0;
}

// What of the row a pass takes: bins lo .. hi, keys key_lo .. key_hi.
struct Range {
    int lo, hi;
    uint32_t key_lo, key_hi;
};

template <class V>
struct Row {
    const V *x;
    int n;
    Lds &s;
    Weights w;

    __device__ __forceinline__ float logit(int i) const
    {
        const float v = (float)x[i] + 0.0f;
        return v == v ? v : -__builtin_inff();
    }

    __device__ __forceinline__ bool takes(const Range &r, float v, uint32_t &key, u64 &weight) const
    {
        int bin;
        key = key_of(v + 0.0f);  // (-0 is 0)
        weight = w.of(v, bin);
        return weight && bin >= r.lo && bin <= r.hi && key >= r.key_lo && key <= r.key_hi;
    }

    // f(i, key, weight) for what a range takes
    template <class F>
    __device__ __forceinline__ void each_of(const Range &r, F f) const
    {
        // (a comparison spares most tokens their weight)
        const float least = w.least(r.hi), most = w.most(r.lo);
        each<4>(x, 0, n, kThreads, [&](int i, float v) {
            uint32_t key;
            u64 weight;
            if (v >= least && v <= most && takes(r, v, key, weight))
                f(i, key, weight);
        });
    }
};

// Of a wave's lanes: the sums up to and with each.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 from_lane(u64 v)
{
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
    return (u64)hi << 32 | lo;
}

__device__ __forceinline__ u64 wave_scan(u64 v)
{
    v += from_lane<0x111, 0xf>(v);  // row_shr:1
    v += from_lane<0x112, 0xf>(v);  // row_shr:2
    v += from_lane<0x114, 0xf>(v);  // row_shr:4
    v += from_lane<0x118, 0xf>(v);  // row_shr:8
    v += from_lane<0x142, 0xa>(v);  // row_bcast:15, into rows 1 and 3
    v += from_lane<0x143, 0xc>(v);  // row_bcast:31, into rows 2 and 3
    return v;
}

// Sums of v over the threads before this one; total: over all.
__device__ u64 scan(Lds &s, u64 v, u64 &total)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const u64 up = wave_scan(v);
    __syncthreads();
    if (lane == 63)
        s.part[wave] = up;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const u64 p = s.part[i];
        before += i < wave ? p : 0;
        total += p;
    }
    return before + up - v;
}

// Sums of `weight` and `count` (kBins of them) become sums of those before each.
__device__ void scan_bins(Lds &s, u64 *weight, uint32_t *count)
{
    const int i = 2 * threadIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const u64 w0 = weight[i], w1 = weight[i + 1];
    const uint32_t n0 = count[i], n1 = count[i + 1];
    const u64 w = wave_scan(w0 + w1), n = wave_scan(n0 + n1);
    u64 *const counts = s.few;  // (not in use yet)
    if (lane == 63) {
        s.part[wave] = w;
        counts[wave] = n;
    }
    __syncthreads();
    u64 before = w - w0 - w1, before_n = n - n0 - n1;
#pragma unroll
    for (int k = 0; k < 16; k++) {
        before += k < wave ? s.part[k] : 0;
        before_n += k < wave ? counts[k] : 0;
    }
    weight[i] = before;
    weight[i + 1] = before + w0;
    count[i] = (uint32_t)before_n;
    count[i + 1] = (uint32_t)before_n + n0;
    if (threadIdx.x == kThreads - 1) {
        weight[kBins] = before + w0 + w1;
        count[kBins] = (uint32_t)before_n + n0 + n1;
    }
    __syncthreads();
}

// A question: the token at which the running weight reaches `weight` (>= 1), or, with a
// count, the count-th.
struct Ask {
    u64 weight;
    uint32_t count;
};

// The bin that holds the answer.
__device__ int find_bin(Lds &s, const Ask &q)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        const bool in = q.count ? s.count[i] < q.count && q.count <= s.count[i + 1]
                                : s.weight[i] < q.weight && q.weight <= s.weight[i + 1];
        if (in)
            s.found_bin = i;
    }
    __syncthreads();
    const int b = s.found_bin;
    __syncthreads();
    return b;
}

// Sorts the first n places of the few, downwards, zeros last; values lie within least ..
// most. Few are ranked by comparing each with all. More are first dealt to 1024 cells of
// equal width in their values, and ranked within those: 1000 in 2.5 us, where compare and
// exchange in 55 steps took 8.
__device__ void sort_few(Lds &s, int n, float least, float most)
{
    constexpr int kCells = kThreads;
    uint32_t *const cell_n = reinterpret_cast<uint32_t *>(s.upto);
    uint32_t *const cell_at = cell_n + kCells;
    const bool cells = n > 256;
    const float per = (float)kCells / (most - least);
    const bool deal = per > 0.0f && per < __builtin_inff();
    u64 mine[2];
    int cell[2], at[2];
    if (cells) {
        cell_n[threadIdx.x] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int i = threadIdx.x + k * kThreads;
        mine[k] = i < n ? s.few[i] : 0;
        if (cells && mine[k]) {
            const float c = (most - value_of((uint32_t)(mine[k] >> 32))) * per;
            cell[k] = deal ? c > 0.0f ? c < kCells - 1 ? (int)c : kCells - 1 : 0 : 0;
            at[k] = (int)atomicAdd(&cell_n[cell[k]], 1u);
        }
    }
    __syncthreads();
    if (cells) {
        u64 total;
        cell_at[threadIdx.x] = (uint32_t)scan(s, cell_n[threadIdx.x], total);
        for (int i = threadIdx.x; i < n; i += kThreads)
            s.few[i] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; k++)
            if (mine[k])
                s.few[cell_at[cell[k]] + at[k]] = mine[k];
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        if (!mine[k])
            continue;
        const int first = cells ? (int)cell_at[cell[k]] : 0;
        const int end = cells ? first + (int)cell_n[cell[k]] : n;
        int rank = first;
        for (int i = first; i < end; i++)
            rank += s.few[i] > mine[k];
        at[k] = rank;
    }
    __syncthreads();
    if (!cells) {
        for (int i = threadIdx.x; i < n; i += kThreads)
            s.few[i] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; k++)
        if (mine[k])
            s.few[at[k]] = mine[k];
    __syncthreads();
}

// Gathers a range's tokens, at most kFew, and sorts them; sums start at base. A comparison
// lets in some of the bins beside the range (at the lowest temperatures many), which are
// taken out again.
template <class V>
__device__ void load_few(const Row<V> &row, const Range &range, u64 base)
{
    Lds &s = row.s;
    if (threadIdx.x == 0)
        s.n = 0;
    for (int i = threadIdx.x; i < kFew; i += kThreads)
        s.few[i] = 0;
    __syncthreads();
    const float least = row.w.least(range.hi), most = row.w.most(range.lo);
    each<8>(row.x, 0, row.n, kThreads, [&](int i, float v) {
        if (v >= least && v <= most) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < (uint32_t)kFew)
                s.few[at] = (u64)key_of(v + 0.0f) << 32 | (uint32_t)~i;
        }
    });
    __syncthreads();
    int let_in = (int)s.n;
    __syncthreads();
    if (threadIdx.x == 0)
        s.n = 0;
    if (let_in > kFew) {
        for (int i = threadIdx.x; i < kFew; i += kThreads)
            s.few[i] = 0;
        __syncthreads();
        row.each_of(range, [&](int i, uint32_t key, u64) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < (uint32_t)kFew)
                s.few[at] = (u64)key << 32 | (uint32_t)~i;
        });
        __syncthreads();
        let_in = (int)s.n < kFew ? (int)s.n : kFew;
        __syncthreads();
        if (threadIdx.x == 0)
            s.n = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < let_in; i += kThreads) {
        uint32_t key;
        u64 weight;
        if (row.takes(range, value_of((uint32_t)(s.few[i] >> 32)), key, weight))
            atomicAdd(&s.n, 1u);
        else
            s.few[i] = 0;
    }
    __syncthreads();
    sort_few(s, let_in, row.w.least(range.hi), fminf(row.w.most(range.lo), (float)row.w.top));
    const int i = 2 * threadIdx.x;
    int bin;
    const u64 w0 = s.few[i] ? row.w.of(value_of((uint32_t)(s.few[i] >> 32)), bin) : 0;
    const u64 w1 = s.few[i + 1] ? row.w.of(value_of((uint32_t)(s.few[i + 1] >> 32)), bin) : 0;
    u64 total;
    const u64 before = base + scan(s, w0 + w1, total);
    s.upto[i] = before + w0;
    s.upto[i + 1] = before + w0 + w1;
    __syncthreads();
}

// The answer among the sorted few, of which base_w and base_n stand before.
__device__ void answer_few(Lds &s, const Ask &q, u64 base_w, uint32_t base_n)
{
    for (int i = threadIdx.x; i < (int)s.n; i += kThreads) {
        const u64 before = i ? s.upto[i - 1] : base_w;
        const bool in = q.count ? base_n + (uint32_t)i + 1 == q.count
                                : before < q.weight && q.weight <= s.upto[i];
        if (in) {
            s.found_w = s.upto[i];
            s.found_id = ~(uint32_t)s.few[i];
        }
    }
    __syncthreads();
}

// The answer within a bin of many tokens.
template <class V>
__device__ __attribute__((noinline)) void answer_many(const Row<V> row, Ask q, int bin, u64 base_w,
                                                      uint32_t base_n)
{
    Lds &s = row.s;
    Range r = {bin, bin, 0, 0xffffffffu};
    // (the bins' sums stay: the ranges' go where the sorted few would)
    u64 *weight = s.few;
    uint32_t *count = reinterpret_cast<uint32_t *>(s.upto);
    // (a turn leaves at most a 512th of the keys: four reach a single one)
    for (int turn = 0; turn < 5; turn++) {
        if (threadIdx.x == 0) {
            s.key_lo = 0xffffffffu;
            s.key_hi = 0;
        }
        __syncthreads();
        uint32_t lo = 0xffffffffu, hi = 0;
        row.each_of(r, [&](int, uint32_t key, u64) {
            lo = key < lo ? key : lo;
            hi = key > hi ? key : hi;
        });
        atomicMin(&s.key_lo, lo);
        atomicMax(&s.key_hi, hi);
        __syncthreads();
        r.key_lo = s.key_lo;
        r.key_hi = s.key_hi;
        __syncthreads();
        if (r.key_lo == r.key_hi)
            break;
        int shift = 0;
        while (((r.key_hi - r.key_lo) >> shift) >= 1024)
            shift++;
        for (int i = threadIdx.x; i < 1024; i += kThreads) {
            weight[i] = 0;
            count[i] = 0;
        }
        __syncthreads();
        row.each_of(r, [&](int, uint32_t key, u64 w) {
            const uint32_t b = (r.key_hi - key) >> shift;
            atomicAdd(&weight[b], w);
            atomicAdd(&count[b], 1u);
        });
        __syncthreads();
        const u64 w0 = weight[threadIdx.x];
        const uint32_t n0 = count[threadIdx.x];
        u64 total;
        const u64 before = base_w + scan(s, w0, total);
        const uint32_t before_n = base_n + (uint32_t)scan(s, n0, total);
        const bool in = q.count ? before_n < q.count && q.count <= before_n + n0
                                : before < q.weight && q.weight <= before + w0;
        if (in) {
            s.found_bin = threadIdx.x;
            s.found_w = before;
            s.found_id = before_n;
            s.n = n0;
        }
        __syncthreads();
        const uint32_t b = (uint32_t)s.found_bin;
        base_w = s.found_w;
        base_n = s.found_id;
        const uint32_t n = s.n;
        __syncthreads();
        r.key_hi -= b << shift;
        const uint32_t span = (1u << shift) - 1u;
        r.key_lo = r.key_hi - r.key_lo > span ? r.key_hi - span : r.key_lo;
        if (n <= (uint32_t)kFew) {
            load_few(row, r, base_w);
            answer_few(s, q, base_w, base_n);
            return;
        }
    }
    // all equal: the place-th by id, each thread counting a run of neighbours
    const int each = (row.n + kThreads - 1) / kThreads;
    const int first = threadIdx.x * each, end = first + each < row.n ? first + each : row.n;
    u64 w1 = 0, w;
    uint32_t n = 0, key;
    for (int i = first; i < end; i++)
        if (row.takes(r, row.logit(i), key, w)) {
            n++;
            w1 = w;
        }
    u64 total;
    const uint32_t before = (uint32_t)scan(s, n, total);
    if (n) {
        const u64 place = q.count ? q.count - base_n : (q.weight - base_w + w1 - 1) / w1;
        if (before < place && place <= before + n) {
            uint32_t left = (uint32_t)place - before;
            for (int i = first; i < end; i++)
                if (row.takes(r, row.logit(i), key, w) && --left == 0)
                    s.found_id = (uint32_t)i;
            s.found_w = base_w + place * w1;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ int part_start(const SampleArgs &g, int part)
{
    return (int)((int64_t)g.V * part / g.parts);
}

// A part's largest logit, the first of equal ones; and the row's sums set to zero.
template <class V>
__global__ __launch_bounds__(kPartThreads) void sample_top_kernel(const SampleArgs g)
{
    __shared__ u64 wave_best[kPartThreads / 64];
    const int t = blockIdx.y, part = blockIdx.x;
    RowSums &row = g.rows[t];
    for (int i = part * kPartThreads + threadIdx.x; i < kBins; i += g.parts * kPartThreads) {
        row.weight[i] = 0;
        row.count[i] = 0;
    }
    if (part == 0 && threadIdx.x == 0)
        row.kept = 0;
    Top own;
    each<4>(static_cast<const V *>(g.logits) + t * g.row_stride, part_start(g, part),
            part_start(g, part + 1), kPartThreads, [&](int i, float v) { own.see(i, v); });
    u64 best = wave_largest(own.packed());
    if ((threadIdx.x & 63) == 0)
        wave_best[threadIdx.x >> 6] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kPartThreads / 64; i++)
            best = largest(best, wave_best[i]);
        row.best[part] = best;
    }
}

// The parts' best as the row's (every thread has it).
__device__ __forceinline__ u64 best_of(const RowSums &row, int parts)
{
    const int lane = threadIdx.x & 63;
    return wave_largest(lane < parts ? row.best[lane] : 0);
}

// A part's bins, added to the row's.
template <class V>
__global__ __launch_bounds__(kPartThreads) void sample_bins_kernel(const SampleArgs g)
{
    __shared__ PartLds s;
    const int t = blockIdx.y, part = blockIdx.x;
    RowSums &row = g.rows[t];
    const float top = value_of((uint32_t)(best_of(row, g.parts) >> 32));
    const Settings set(g, t);
    if (set.first || top == -__builtin_inff())
        return;
    fill_powers(s.power, kPartThreads);
    for (int i = threadIdx.x; i < kBins; i += kPartThreads) {
        s.weight[i] = 0;
        s.count[i] = 0;
    }
    if (threadIdx.x == 0)
        s.kept = 0;
    Weights w;
    w.set(s.power, top, set.heat);
    __syncthreads();
    const u64 kept = fill_bins(static_cast<const V *>(g.logits) + t * g.row_stride,
                               part_start(g, part), part_start(g, part + 1), kPartThreads, w,
                               s.weight, s.count, set);
    atomicAdd(&s.kept, kept);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kPartThreads)
        if (s.weight[i]) {
            atomicAdd(&row.weight[i], s.weight[i]);
            if (set.k > 0)
                atomicAdd(&row.count[i], s.count[i]);
        }
    if (threadIdx.x == 0)
        atomicAdd(&row.kept, s.kept);
}

// SHARED: the launches above have the row's best and bins.
template <class V, bool SHARED>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs g)
{
    extern __shared__ __attribute__((aligned(16))) char mem[];
    Lds &s = *reinterpret_cast<Lds *>(mem);
    const int t = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    Row<V> row = {static_cast<const V *>(g.logits) + t * g.row_stride, g.V, s, {}};
    const Settings set(g, t);

    // the largest logit, the first of equal ones
    u64 best = 0;
    if constexpr (SHARED) {
        best = best_of(g.rows[t], g.parts);
    } else {
        Top own;
        each<8>(row.x, 0, g.V, kThreads, [&](int i, float v) { own.see(i, v); });
        best = wave_largest(own.packed());
        if (lane == 0)
            s.part[wave] = best;
        __syncthreads();
        for (int i = 0; i < 16; i++)
            best = largest(best, s.part[i]);
    }
    const float top = value_of((uint32_t)(best >> 32));
    const bool none = top == -__builtin_inff();
    if (none || set.first) {
        if (threadIdx.x == 0) {
            g.tokens[t] = none ? -1 : (int32_t)~(uint32_t)best;
            if (g.logprobs)
                g.logprobs[t] = none ? -__builtin_inff() : 0.0f;
        }
        return;
    }

    if (threadIdx.x == 0) {  // (answers stay in bounds, also for logits that change meanwhile)
        s.found_bin = 0;
        s.found_id = 0;
        s.found_w = (u64)kOne;
    }
    fill_powers(s.power, kThreads);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.weight[i] = SHARED ? g.rows[t].weight[i] : 0;
        s.count[i] = SHARED ? g.rows[t].count[i] : 0;
    }
    row.w.set(s.power, top, set.heat);
    __syncthreads();
    u64 left;  // what min_p leaves, then all filters
    if constexpr (SHARED) {
        left = g.rows[t].kept;
    } else {
        const u64 kept = fill_bins(row.x, 0, g.V, kThreads, row.w, s.weight, s.count, set);
        scan(s, kept, left);
    }
    if (set.k <= 0)
        for (int i = threadIdx.x; i < kBins; i += kThreads)
            s.count[i] = most_tokens(s.weight[i], i, s.power);
    __syncthreads();
    scan_bins(s, s.weight, s.count);

    // top_k, top_p and the draw, each asked where it says anything; `all` is what top_k and
    // top_p leave, `left` what min_p does, then all three. The sorted few: bins lo .. hi, if any.
    int lo = 0, hi = -1;
    u64 all = s.weight[kBins];
    for (int turn = 0; turn < 3; turn++) {
        Ask q = {0, 0};
        if (turn == 0) {
            if (set.k <= 0 || (uint32_t)set.k >= s.count[kBins])
                continue;
            q.count = (uint32_t)set.k;
        } else if (turn == 1) {
            if (!(set.p < 1.0f))
                continue;
            q.weight = (u64)ceil((double)set.p * (double)all);
            q.weight = q.weight < 1 ? 1 : q.weight > all ? all : q.weight;
        } else {
            float u = g.u[t];
            u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;  // (the product stays below 2^64)
            left = set.floor > 0.0f && left < all ? left : all;
            q.weight = (u64)((double)u * (double)left) + 1;
            q.weight = q.weight > left ? left : q.weight;
        }
        const int b = find_bin(s, q);
        if ((b < lo || b > hi) && s.count[b + 1] - s.count[b] > (uint32_t)kFew) {
            lo = 0;
            hi = -1;  // (the few's memory is used for the search)
            answer_many(row, q, b, s.weight[b], s.count[b]);
        } else {
            if (b < lo || b > hi) {
                lo = turn < 2 && s.count[b + 1] <= (uint32_t)kFew ? 0 : b;
                hi = b;
                load_few(row, Range{lo, hi, 0, 0xffffffffu}, s.weight[lo]);
            }
            answer_few(s, q, s.weight[lo], s.count[lo]);
        }
        if (turn < 2)
            all = s.found_w;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const uint32_t id = s.found_id;
        g.tokens[t] = (int32_t)id;
        if (g.logprobs) {
            const float v = row.logit((int)id);
            const double e = row.w.infinite ? 0.0 : ((double)v - (double)top) / (double)set.heat;
            g.logprobs[t] = (float)(e - log((double)left / kOne));
        }
    }
}

template <class V>
int launch(const SampleArgs &g, int64_t T, hipStream_t stream)
{
    auto row = [&](auto *kernel) {
        allow_dynamic_lds(reinterpret_cast<const void *>(kernel), sizeof(Lds));
        hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(kThreads), sizeof(Lds), stream, g);
        return check_launch();
    };
    if (g.parts == 1)
        return row(sample_kernel<V, false>);
    const dim3 grid((unsigned)g.parts, (unsigned)T);
    hipLaunchKernelGGL((sample_top_kernel<V>), grid, dim3(kPartThreads), 0, stream, g);
    if (int rc = check_launch())
        return rc;
    hipLaunchKernelGGL((sample_bins_kernel<V>), grid, dim3(kPartThreads), 0, stream, g);
    if (int rc = check_launch())
        return rc;
    return row(sample_kernel<V, true>);
}

// Workgroups that share a row: as many as give the device 512, of 2048 logits at least, where
// that is faster than its own alone, which spares two launches. Measured over 1 to 192 rows of
// 4096 to 1000000 logits, the border runs from 45000 logits (one row: 30 us alone, 27 shared,
// of 50000; 25 and 27 of 32001) by 64000 (32 rows: 43 and 41) to 131071 (128 rows: 75 and 71;
// 69 and 74 of 100003).
constexpr int64_t kSharedRows = 128;

// The most rows that are shared, of V logits.
int64_t shared_rows(int64_t V) { return V < 40000 ? 0 : std::min((V - 40000) / 700, kSharedRows); }

int parts_of(int64_t T, int64_t V)
{
    if (T < 1 || T > shared_rows(V))
        return 1;
    return (int)std::min<int64_t>({512 / T, V / 2048, kPartsMax});
}

}  // namespace

// What the largest call of up to T rows needs, so that a workspace serves smaller calls too (more
// rows than are shared need none themselves).
size_t sample_workspace(int64_t T, int64_t V)
{
    return ((size_t)std::min(T, shared_rows(V)) * sizeof(RowSums) + 255) / 256 * 256;
}

int launch_sample(const void *logits, int64_t row_stride, const float *temperature,
                  const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                  int32_t *tokens, float *logprobs, int64_t T, int64_t V, int dtype,
                  void *workspace, hipStream_t stream)
{
    const SampleArgs g = {logits, row_stride, temperature, top_k, top_p, min_p, u, tokens, logprobs,
                          static_cast<RowSums *>(workspace), (int)V, parts_of(T, V)};
    if (dtype == BQM_DTYPE_F32)
        return launch<float>(g, T, stream);
    if (dtype == BQM_DTYPE_F16)
        return launch<_Float16>(g, T, stream);
    return launch<__bf16>(g, T, stream);
}

}  // namespace bqm
