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
#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kFew = 2048;  // tokens that are sorted in LDS
constexpr int kSteps = 1024;  // of the table of powers, in a factor of 2
constexpr double kOne = 17592186044416.0;  // 2^44

struct SampleArgs {
    const void *logits;
    int64_t row_stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *tokens;
    float *logprobs;
    int V;
};

struct Lds {
    double power[kSteps];      // 2^(i / kSteps)
    u64 weight[kBins + 1];     // sums of the bins before each
    uint32_t count[kBins + 1];
    u64 few[kFew];             // key << 32 | ~id, sorted downwards
    u64 upto[kFew];            // weights of those up to and with each
    u64 part[16];
    uint32_t part_n[16];
    u64 found_w;               // an answer: the weights up to and with the token,
    uint32_t found_id;         // the token,
    int found_bin;
    uint32_t n, key_lo, key_hi;
};

template <class V>
__device__ __forceinline__ float logit(const V *x, int i)
{
    const float v = (float)x[i] + 0.0f;  // (-0 is 0)
    return v == v ? v : -__builtin_inff();
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

// A logit's weight, a whole number of 2^-44, and bin.
struct Weights {
    const double *power;
    double top, c;  // the largest logit; kSteps * log2(e) / temperature
    bool infinite;

    __device__ __forceinline__ u64 of(float v, int &bin) const
    {
        bin = 0;
        if (infinite)
            return v == __builtin_inff() ? (u64)kOne : 0;
        const double y = ((double)v - top) * c;
        if (!(y > -46.0 * kSteps))
            return 0;
        const double f = floor(y);
        const int k = (int)f;
        bin = (-k) >> 5;
        // 2^(y / kSteps) = power of the whole part times e^r, r below 2^-10: the series'
        // third power leaves 2^-46, its fp32 rounding 2^-34
        const float r = (float)(y - f) * 6.7690154351557158e-4f;  // ln(2) / kSteps
        const float p = r * fmaf(r, fmaf(r, 0.16666667f, 0.5f), 1.0f);
        double w = power[k & (kSteps - 1)];
        w = __builtin_fma(w, (double)p, w);
        // in 2^52 .. 2^53 a double's last bit is 1: the sum rounds to a whole number
        w = ldexp(w, 44 + (k >> 10)) + 4503599627370496.0;
        return (u64)__double_as_longlong(w) & 0xfffffffffffffull;
    }
};

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

    __device__ __forceinline__ bool takes(const Range &r, int i, uint32_t &key, u64 &weight) const
    {
        const float v = logit(x, i);
        int bin;
        key = key_of(v);
        weight = w.of(v, bin);
        return weight && bin >= r.lo && bin <= r.hi && key >= r.key_lo && key <= r.key_hi;
    }
};

// Sums of v over the threads before this one; total: over all.
__device__ u64 scan(Lds &s, u64 v, u64 &total)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    u64 up = v;
    for (int m = 1; m < 64; m <<= 1) {
        const u64 o = __shfl_up(up, m, 64);
        if (lane >= m)
            up += o;
    }
    __syncthreads();
    if (lane == 63)
        s.part[wave] = up;
    __syncthreads();
    u64 before = 0;
    total = 0;
    for (int i = 0; i < 16; i++) {
        if (i < wave)
            before += s.part[i];
        total += s.part[i];
    }
    return before + up - v;
}

// Sums of `weight` and `count` (kBins of them) become sums of those before each.
__device__ void scan_bins(Lds &s, u64 *weight, uint32_t *count)
{
    const int i = 2 * threadIdx.x;
    const u64 w0 = weight[i], w1 = weight[i + 1];
    const uint32_t n0 = count[i], n1 = count[i + 1];
    u64 total, total_n;
    const u64 before = scan(s, w0 + w1, total);
    const u64 before_n = scan(s, n0 + n1, total_n);
    weight[i] = before;
    weight[i + 1] = before + w0;
    count[i] = (uint32_t)before_n;
    count[i + 1] = (uint32_t)before_n + n0;
    if (threadIdx.x == 0) {
        weight[kBins] = total;
        count[kBins] = (uint32_t)total_n;
    }
    __syncthreads();
}

// A question: the token at which the running weight reaches `weight` (>= 1), or, with a
// count, the count-th.
struct Ask {
    u64 weight;
    uint32_t count;
};

// The place among `bins` sums that holds the answer, given base before the first.
__device__ int find_bin(Lds &s, const Ask &q, u64 base_w, uint32_t base_n)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        const bool in = q.count ? base_n + s.count[i] < q.count && q.count <= base_n + s.count[i + 1]
                                : base_w + s.weight[i] < q.weight &&
                                      q.weight <= base_w + s.weight[i + 1];
        if (in)
            s.found_bin = i;
    }
    __syncthreads();
    const int b = s.found_bin;
    __syncthreads();
    return b;
}

// Gathers a range's tokens (at most kFew) and sorts them; sums start at base.
template <class V>
__device__ void load_few(const Row<V> &row, const Range &range, u64 base)
{
    Lds &s = row.s;
    if (threadIdx.x == 0)
        s.n = 0;
    for (int i = threadIdx.x; i < kFew; i += kThreads)
        s.few[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        uint32_t key;
        u64 weight;
        if (row.takes(range, i, key, weight)) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < (uint32_t)kFew)
                s.few[at] = (u64)key << 32 | (uint32_t)~i;
        }
    }
    __syncthreads();
    int p = 2;
    while (p < (int)s.n)
        p <<= 1;
    for (int size = 2; size <= p; size <<= 1)
        for (int step = size >> 1; step; step >>= 1) {
            const int i = threadIdx.x;  // pairs: at most 1024
            if (i < p / 2) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const u64 u = s.few[a], v = s.few[b];
                if ((u < v) == ((a & size) == 0)) {
                    s.few[a] = v;
                    s.few[b] = u;
                }
            }
            __syncthreads();
        }
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
__device__ void answer_many(const Row<V> &row, const Ask &q, int bin, u64 base_w, uint32_t base_n)
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
        for (int i = threadIdx.x; i < row.n; i += kThreads) {
            uint32_t key;
            u64 w;
            if (row.takes(r, i, key, w)) {
                lo = key < lo ? key : lo;
                hi = key > hi ? key : hi;
            }
        }
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
        for (int i = threadIdx.x; i < row.n; i += kThreads) {
            uint32_t key;
            u64 w;
            if (row.takes(r, i, key, w)) {
                const uint32_t b = (r.key_hi - key) >> shift;
                atomicAdd(&weight[b], w);
                atomicAdd(&count[b], 1u);
            }
        }
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
        if (row.takes(r, i, key, w)) {
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
                if (row.takes(r, i, key, w) && --left == 0)
                    s.found_id = (uint32_t)i;
            s.found_w = base_w + place * w1;
        }
    }
    __syncthreads();
}

template <class V>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs g)
{
    extern __shared__ __attribute__((aligned(16))) char mem[];
    Lds &s = *reinterpret_cast<Lds *>(mem);
    const int t = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    Row<V> row = {static_cast<const V *>(g.logits) + t * g.row_stride, g.V, s, {}};

    // the largest logit, the first of equal ones
    u64 best = 0;
    for (int i = threadIdx.x; i < g.V; i += kThreads) {
        const u64 k = (u64)key_of(logit(row.x, i)) << 32 | (uint32_t)~i;
        best = k > best ? k : best;
    }
    for (int m = 32; m; m >>= 1) {
        const u64 o = __shfl_xor(best, m, 64);
        best = o > best ? o : best;
    }
    if (lane == 0)
        s.part[wave] = best;
    __syncthreads();
    for (int i = 0; i < 16; i++)
        best = s.part[i] > best ? s.part[i] : best;
    const float top = value_of((uint32_t)(best >> 32));
    const float heat = g.temperature ? g.temperature[t] : 1.0f;
    const int k = g.top_k ? g.top_k[t] : 0;
    const float p = g.top_p ? g.top_p[t] : 1.0f;
    const float floor_p = g.min_p ? g.min_p[t] : 0.0f;
    const bool none = top == -__builtin_inff();
    // (written so that NaN settings take the first token)
    if (none || !(heat > 0.0f) || k == 1 || !(p > 0.0f) || !(floor_p <= 1.0f)) {
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
    for (int i = threadIdx.x; i < kSteps; i += kThreads)
        s.power[i] = exp2((double)i / kSteps);
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.weight[i] = 0;
        s.count[i] = 0;
    }
    row.w.power = s.power;
    row.w.top = top;
    row.w.infinite = top == __builtin_inff();
    row.w.c = kSteps * 1.4426950408889634 / (double)heat;
    __syncthreads();

    // counts and weights of the bins, and the weights that min_p leaves
    const double least = (double)floor_p * kOne;
    u64 kept = 0;
    for (int i = threadIdx.x; i < g.V; i += kThreads) {
        int bin;
        const u64 w = row.w.of(logit(row.x, i), bin);
        if (w) {
            atomicAdd(&s.weight[bin], w);
            atomicAdd(&s.count[bin], 1u);
            if ((double)w >= least)
                kept += w;
        }
    }
    __syncthreads();
    scan_bins(s, s.weight, s.count);
    u64 left;
    scan(s, kept, left);

    // the sorted few: bins lo .. hi, if any
    int lo = 0, hi = -1;
    auto ask = [&](const Ask &q, bool last) {
        const int b = find_bin(s, q, 0, 0);
        if (b < lo || b > hi) {
            if (s.count[b + 1] - s.count[b] > (uint32_t)kFew) {
                lo = 0;
                hi = -1;  // (the few's memory is used for the search)
                answer_many(row, q, b, s.weight[b], s.count[b]);
                return;
            }
            lo = !last && s.count[b + 1] <= (uint32_t)kFew ? 0 : b;
            hi = b;
            load_few(row, Range{lo, hi, 0, 0xffffffffu}, s.weight[lo]);
        }
        answer_few(s, q, s.weight[lo], s.count[lo]);
    };
    u64 all = s.weight[kBins];
    if (k > 0 && (uint32_t)k < s.count[kBins]) {
        ask(Ask{0, (uint32_t)k}, false);
        all = s.found_w;
        __syncthreads();
    }
    left = left < all ? left : all;
    if (p < 1.0f) {
        const u64 need = (u64)ceil((double)p * (double)all);
        ask(Ask{need < 1 ? 1 : need > all ? all : need, 0}, false);
        left = s.found_w < left ? s.found_w : left;
        __syncthreads();
    }
    float u = g.u[t];
    u = u > 0.0f ? u : 0.0f;
    const u64 at = (u64)((double)u * (double)left) + 1;
    ask(Ask{at > left ? left : at, 0}, true);
    if (threadIdx.x == 0) {
        const uint32_t id = s.found_id;
        g.tokens[t] = (int32_t)id;
        if (g.logprobs) {
            const float v = logit(row.x, (int)id);
            const double e = row.w.infinite ? 0.0 : ((double)v - (double)top) / (double)heat;
            g.logprobs[t] = (float)(e - log((double)left / kOne));
        }
    }
}

template <class V>
int launch(const SampleArgs &g, int64_t T, hipStream_t stream)
{
    allow_dynamic_lds(reinterpret_cast<const void *>(sample_kernel<V>), sizeof(Lds));
    hipLaunchKernelGGL((sample_kernel<V>), dim3((unsigned)T), dim3(kThreads), sizeof(Lds), stream,
                       g);
    return check_launch();
}

}  // namespace

size_t sample_workspace(int64_t, int64_t) { return 0; }

int launch_sample(const void *logits, int64_t row_stride, const float *temperature,
                  const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                  int32_t *tokens, float *logprobs, int64_t T, int64_t V, int dtype, void *,
                  hipStream_t stream)
{
    const SampleArgs g = {logits, row_stride, temperature, top_k, top_p, min_p,
                          u,      tokens,     logprobs,    (int)V};
    if (dtype == BQM_DTYPE_F32)
        return launch<float>(g, T, stream);
    if (dtype == BQM_DTYPE_F16)
        return launch<_Float16>(g, T, stream);
    return launch<__bf16>(g, T, stream);
}

}  // namespace bqm
