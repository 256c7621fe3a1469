// attention.hip -- attention of new tokens over a paged cache.
//
// out = sum_j e_j v_j / sum_j e_j, e_j = exp(scale q.k_j - max): one pass over
// the keys with the running maximum and sum of each row.
//
// Rows. The query heads of one key/value head see the same keys, so a row is a
// (token, head of the group) pair: row r of a sequence is token r / group, head
// r % group, and 32 rows share every key tile a wave reads. A single token with
// 4 heads fills 4 of 32 rows; the matrix cores have that to spare while the
// cache streams from memory.
//
// Matrix products, transposed so that a row of the softmax lies in one lane
// pair (l, l + 32): S^T = K Q^T (32 tokens x 32 rows, 32x32x16 products), lane l
// holding row l % 32 of 16 tokens; then O^T += V^T P^T takes P^T from the same
// registers: the product's k index may name tokens in any order, and the order
// in which a lane holds its scores (4 of 8 tokens each half) is also the one in
// which a transposing LDS read delivers V.
//
// What bounds it, measured on one MI355X (bf16, heads of 128, 32 over 8):
//   one token a sequence: memory. 64 sequences of 4096 tokens 202 us (5.3 TB/s; a
//     large copy reaches 5.0), of 16384 784 us (5.5 TB/s); 64 of 33 to 8192 tokens
//     105 us (4.2 TB/s), 2 of about 120000 177 us (5.4 TB/s).
//   a prompt of 8192: issue and the workgroups' ends. 559 us, 985 TFLOP/s where a
//     large matrix product of the library reaches 1380; matrix units 44% busy, the
//     vector unit's softmax beside them, 61 us of start and end of 1024 workgroups.
//   chunks of 17 sequences, heads of 64, a window of 1024: 40 us; uneven shares (572
//     workgroups, three a compute unit) and waits, matrix units 15% busy.
//   one token over 37: latency, 8 us of which an empty launch is 4.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mfma(f16x8 a, f16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <class T>
struct Operand;
template <>
struct Operand<_Float16> {
    typedef f16x8 type;
};
template <>
struct Operand<__bf16> {
    typedef bf16x8 type;
};

struct AttnArgs {
    const void *q;
    const u32x4 *k, *v;  // 16-byte pieces of 8 values
    void *out;
    const int32_t *pages, *kv_lens, *q_starts;
    float *part;         // [n_splits][total_q][n_q_heads][dim], unscaled sums
    float2 *part_ml;     // the same rows' maximum (log2) and sum of weights
    int64_t q_token, q_head, pages_stride, total_q;
    uint32_t c_page, c_token, c_head;  // strides in pieces
    uint32_t span;       // bytes of one head's pieces, first to last; 0: 4 GiB or more
    int n_pages, n_seqs, max_pages, page_size, max_kv;
    int n_q_heads, n_heads, group, dim;
    int tiles, n_splits, chunk;
    float scale_log2;    // scale * log2(e)
    int causal, window;
};

// What invalid pieces (tokens past the range, values past the head) are read
// from: zeros, so that no stale value, NaN included, meets a product.
__device__ const u32x4 kZeros = {0, 0, 0, 0};

typedef const __attribute__((address_space(1))) u32x4 *piece_ptr;

// In the place of a token that there is none of, in pieces: behind every span below
// 4 GiB, with any piece of a head added; and where places need all 32 bits.
constexpr uint32_t kNoPlace = 0x0fffff00u, kNoWidePlace = 0xffffffffu;

// The kernel's steps are lambdas called from several places; left to itself the
// compiler makes calls of some, with the registers they share in memory.
#define BQM_INLINE __attribute__((always_inline))

// A tile of rows: its sequence, and the tokens that any of its rows sees.
struct Tile {
    int seq, tile;      // tile of the sequence
    int64_t q0;         // the sequence's first token row
    int q_len, rows;    // its tokens and (token, head) rows
    int kv_len;
    int begin, end;     // tokens seen
};

__device__ __forceinline__ int row_lo(const AttnArgs &a, int pos)
{
    return a.window > 0 ? (int)max((int64_t)0, (int64_t)pos - a.window + 1) : 0;
}

__device__ __forceinline__ int row_hi(const AttnArgs &a, int kv_len, int pos)
{
    return a.causal ? min(kv_len, pos + 1) : kv_len;
}

__device__ __forceinline__ void sequence_of(const AttnArgs &a, int b, int start, int next,
                                            int len, Tile &t)
{
    t.seq = b;
    t.q0 = min(max((int64_t)start, (int64_t)0), a.total_q);
    t.q_len = (int)min(max((int64_t)next - t.q0, (int64_t)0), a.total_q - t.q0);
    t.rows = t.q_len * a.group;
    const int64_t room = min((int64_t)a.max_pages * a.page_size, (int64_t)a.max_kv);
    t.kv_len = (int)min((int64_t)max(len, 0), room);
}

__device__ __forceinline__ void load_sequence(const AttnArgs &a, int b, Tile &t)
{
    // the same in all lanes: kept in scalar registers
    sequence_of(a, b, __builtin_amdgcn_readfirstlane(a.q_starts[b]),
                __builtin_amdgcn_readfirstlane(a.q_starts[b + 1]),
                __builtin_amdgcn_readfirstlane(a.kv_lens[b]), t);
}

template <int M>
__device__ __forceinline__ void load_range(const AttnArgs &a, Tile &t)
{
    const int first = t.tile * M / a.group;
    const int last = min(t.tile * M + M - 1, t.rows - 1) / a.group;
    const int base = t.kv_len - t.q_len;
    t.begin = row_lo(a, base + first);
    t.end = row_hi(a, t.kv_len, base + last);
}

// How many parts the tile's tokens are cut into: at most n_splits, since n_splits
// chunks hold the most tokens that a tile's rows can see.
__device__ __forceinline__ int parts_of(const AttnArgs &a, const Tile &t)
{
    return a.n_splits > 1 && t.end - t.begin > a.chunk
               ? (t.end - t.begin + a.chunk - 1) / a.chunk
               : 1;
}

// The last sequence b for which first(q_starts[b], b) <= x (first ascends with
// b, and that of sequence 0 is not above x). All lanes take part: each step
// narrows the range to a 64th, one load's latency instead of six bisections'.
template <class First>
__device__ __forceinline__ int find_sequence(const AttnArgs &a, int64_t x, First first)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.n_seqs;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int b = lo + lane * step;
        const bool in = lane * step < n && first(a.q_starts[min(b, a.n_seqs - 1)], b) <= x;
        const int k = max(__popcll(__ballot(in)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Tile x of the launch. Sequence b's tiles start at floor(q_starts[b] * group /
// M) + b: never fewer places than it has tiles, some left empty, and found
// without a table of sums.
template <int M>
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int x, Tile &t)
{
    auto first = [&](int start, int b) { return (int64_t)start * a.group / M + b; };
    const int b = find_sequence(a, x, first);
    load_sequence(a, b, t);
    t.tile = x - (int)first(__builtin_amdgcn_readfirstlane(a.q_starts[b]), b);
    if (t.tile < 0 || (int64_t)t.tile * M >= t.rows)
        return false;
    load_range<M>(a, t);
    return true;
}

// Piece x of a launch of few rows: (tile, part) pairs that exist come first, whole
// chunks before what they leave over, so that sequences of very different lengths
// fill the card evenly and the places of pieces that do not exist come when all
// others are under way. A lane counts a sequence's pieces, in groups of 64.
constexpr int kCountedSeqs = 128;

__device__ __forceinline__ int wave_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        v += lane >= d ? u : 0;
    }
    return v;
}

template <int M>
__device__ __forceinline__ bool find_piece(const AttnArgs &a, int x, Tile &t, int &part)
{
    constexpr int kGroups = kCountedSeqs / 64;
    const int lane = threadIdx.x & 63;
    int tiles[kGroups], whole[kGroups], tiles_upto[kGroups], whole_upto[kGroups];
    int n_whole = 0;
#pragma unroll
    for (int g = 0; g < kGroups; g++) {
        const int b = g * 64 + lane, bc = min(b, a.n_seqs - 1);
        Tile s;
        sequence_of(a, bc, a.q_starts[bc], a.q_starts[bc + 1], a.kv_lens[bc], s);
        tiles[g] = b < a.n_seqs && s.rows > 0 ? (s.rows - 1) / M + 1 : 0;
        // by the widest any tile could be: a part too many is found empty later
        const int base = s.kv_len - s.q_len;
        const int seen = row_hi(a, s.kv_len, s.kv_len - 1) - row_lo(a, base);
        whole[g] = seen > a.chunk ? tiles[g] * ((seen + a.chunk - 1) / a.chunk - 1) : 0;
        tiles_upto[g] = wave_scan(tiles[g]);
        whole_upto[g] = n_whole + wave_scan(whole[g]);
        n_whole = __builtin_amdgcn_readlane(whole_upto[g], 63);
    }
    const bool left_over = x >= n_whole;
    if (left_over)
        x -= n_whole;
    int before = 0;
#pragma unroll
    for (int g = 0; g < kGroups; g++) {
        const int n = left_over ? tiles[g] : whole[g];
        const int upto = left_over ? before + tiles_upto[g] : whole_upto[g];
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (x < all) {
            const int k = __popcll(__ballot(upto <= x));
            load_sequence(a, g * 64 + k, t);
            const int i = x - (__builtin_amdgcn_readlane(upto, k) - __builtin_amdgcn_readlane(n, k));
            const int n_tiles = __builtin_amdgcn_readlane(tiles[g], k);
            t.tile = i % n_tiles;
            part = left_over ? 0 : 1 + i / n_tiles;
            load_range<M>(a, t);
            return true;
        }
        before = all;
    }
    return false;
}

// Maximum and sum over a lane pair (l, l + 32): the two halves of a softmax row.
__device__ __forceinline__ float pair_max(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float pair_sum(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The finite ones of eight values, the others as zeros.
template <class T>
__device__ __forceinline__ u32x4 finite_only(u32x4 v)
{
    constexpr short e = __is_same(T, _Float16) ? 0x7c00 : 0x7f80;  // the exponent's bits
    const s16x8 w = __builtin_bit_cast(s16x8, v);
    return __builtin_bit_cast(u32x4, w & ((w & e) != e));
}

template <class O>
__device__ __forceinline__ void store4(O *p, f32x4 v)
{
    typedef O o4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<o4 *>(p) = __builtin_convertvector(v, o4);
}

// WM waves share a key tile, 32 rows each; WK such groups take every WK-th tile
// of 32 * NT tokens and are joined at the end.
template <int DP, int WM, int WK, int NT>
struct Shape {
    static constexpr int M = 32 * WM;
    static constexpr int kThreads = 64 * WM * WK;
    static constexpr int TK = 32 * NT;
    static constexpr int kPieces = DP / 8;                     // of a row
    static constexpr int kLoads = TK * kPieces / (64 * WM);    // a thread's, of K and of V
    static constexpr int kRowsPerLoad = 64 * WM / kPieces;
    // LDS rows are padded: K by 16 bytes (neighbouring lanes read 16 bytes of
    // neighbouring rows), V by 64 (32 lanes read 64 bytes of 4 rows), so that no two
    // of them share one of the 64 banks: no conflicts counted
    static constexpr int KS = DP * 2 + 16, VS = DP * 2 + 64;
    static constexpr int kTile = TK * (KS + VS);
    static constexpr int kBufs = WM > 1 ? 2 : 1;
    static constexpr int kStage = kTile * kBufs * WK;
    static constexpr int kJoin = WK > 1 ? WK * (DP / 32) * 4096 + WK * 256 : 0;
    static constexpr int kLds = kStage > kJoin ? kStage : kJoin;
};

// WAVES: a SIMD's. With eight waves the workgroup is two halves out of step: while
// the four waves of one (one a SIMD) are at their matrix products, the others are
// at their softmax, and a barrier has them change places (prompt of 8192: 571 us;
// two workgroups of four waves a compute unit, left to fall out of step by
// themselves, 608). A wave with 64 rows would read half as much from LDS, but
// its scores then come to lie in accumulator registers and are moved one by one:
// 1040 us.
template <class T, class O, int DP, int WM, int WK, int NT, int WAVES>
__global__ __launch_bounds__(64 * WM *WK, WAVES) void attention_kernel(AttnArgs a)
{
    typedef Shape<DP, WM, WK, NT> S;
    typedef typename Operand<T>::type Op;
    typedef f32x16 Scores[NT];
    constexpr bool kHalves = WM == 8;
    extern __shared__ char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wk = wave / WM;
    const int half = lane >> 5, col = lane & 31;

    // heads lie next to one another in the grid, so that with eight of them each
    // XCD's L2 holds one head's keys and values; causal tiles go longest first
    int x = blockIdx.x;
    const int head = x % a.n_heads;
    x /= a.n_heads;
    Tile t;
    int split;
    if (WK > 1 && a.n_splits > 1 && a.n_seqs <= kCountedSeqs) {
        if (!find_piece<S::M>(a, x, t, split))
            return;
    } else {
        split = a.n_splits - 1 - x / a.tiles;
        if (!find_tile<S::M>(a, a.tiles - 1 - x % a.tiles, t))
            return;
    }
    const int parts = kHalves ? 1 : parts_of(a, t);  // tiles of 256 rows are not cut
    if (split >= parts)
        return;
    // part 0 is what whole chunks leave over; it goes last, and fills the gaps that
    // the whole ones leave on the card
    const int c1 = t.end - (parts - 1 - split) * a.chunk;
    const int c0 = split == 0 ? t.begin : c1 - a.chunk;

    // this lane's row; rows past the end repeat the last and store nothing
    const int row_first = t.tile * S::M + wm * 32;
    const int rc = min(row_first + col, t.rows - 1);
    const int tok = rc / a.group, g = rc - tok * a.group;
    const int pos = t.kv_len - t.q_len + tok;
    const int lo = max(row_lo(a, pos), c0), hi = min(row_hi(a, t.kv_len, pos), c1);
    // rows ascend with the lanes, and so do lo and hi
    const int lo_first = __builtin_amdgcn_readlane(lo, 0);
    const int lo_last = __builtin_amdgcn_readlane(lo, 31);
    const int hi_first = __builtin_amdgcn_readlane(hi, 0);
    const int hi_last = __builtin_amdgcn_readlane(hi, 31);
    const int64_t q_row = t.q0 + tok;
    const int q_head = head * a.group + g;
    const int64_t out_row = q_row * a.n_q_heads + q_head;
    Op qf[DP / 16];
    {
        const T *qp = static_cast<const T *>(a.q) + q_row * a.q_token + q_head * a.q_head;
#pragma unroll
        for (int kk = 0; kk < DP / 16; kk++) {
            const int d = 16 * kk + 8 * half;
            const T *p = d < a.dim ? qp + d : reinterpret_cast<const T *>(&kZeros);
            qf[kk] = *reinterpret_cast<const Op *>(p);
        }
    }

    // ---- staging: this group's tiles are n = 0, 1, ..: tokens t0(n) = c0 + (n WK + wk) TK
    const int iters = (c1 - c0 + WK * S::TK - 1) / (WK * S::TK);
    const int t00 = c0 + wk * S::TK;
    const int gt = wm * 64 + lane;  // thread of the group
    const int piece = gt % S::kPieces, row0 = gt / S::kPieces;
    const bool piece_ok = piece * 8 < a.dim;
    // Pieces are read through buffer resources of the head's span: a place behind
    // its end reads as zeros without a branch. Caches of 4 GiB and more a layer,
    // beyond a resource's offsets, are read through pointers.
    const u32x4 *const kh = a.k + (uint64_t)head * a.c_head, *const vh = a.v + (uint64_t)head * a.c_head;
    const __amdgpu_buffer_rsrc_t kb_rsrc = make_rsrc(kh, a.span), vb_rsrc = make_rsrc(vh, a.span);
    const uint32_t none = a.span != 0 ? kNoPlace : kNoWidePlace;
    char *const buf = lds + wk * S::kTile * S::kBufs;
    auto k_of = [&](int n) { return buf + (S::kBufs > 1 ? n & 1 : 0) * S::kTile; };
    auto v_of = [&](int n) { return k_of(n) + S::TK * S::KS; };
    const int32_t *table = a.pages + t.seq * a.pages_stride;

    // lane l looks up token l of the tile to be read next; page and place advance
    // by a tile at a time without a division. (The look-up goes out before a tile's
    // loads: loads are waited for in order, so one behind them would take their time.)
    const int step_page = WK * S::TK / a.page_size, step_place = WK * S::TK % a.page_size;
    int ct, cpage, cplace, page_id, place;
    const int last_page = max(c1 - 1, 0) / a.page_size;
    auto look_up = [&]() BQM_INLINE {
        page_id = table[min(cpage, last_page)];
        place = ct < c1 ? cplace : -1;
        ct += WK * S::TK;
        cpage += step_page;
        cplace += step_place;
        const bool over = cplace >= a.page_size;
        cplace -= over ? a.page_size : 0;
        cpage += over;
    };
    // of lane l's token, in pieces
    auto place_of = [&]() BQM_INLINE {
        const uint32_t at = (uint32_t)page_id * a.c_page + (uint32_t)place * a.c_token;
        return place >= 0 && (uint32_t)page_id < (uint32_t)a.n_pages ? at : none;
    };
    // this thread's rows' places
    typedef uint32_t Places[S::kLoads];
    auto spread = [&](Places &of, uint32_t mine) BQM_INLINE {
#pragma unroll
        for (int i = 0; i < S::kLoads; i++)
            of[i] = __shfl(mine, row0 + i * S::kRowsPerLoad, 64);
    };
    u32x4 kr[S::kLoads], vr[S::kLoads];
    // piece i of the thread's; none of a head's values beyond its own
    auto load = [&](const u32x4 *base, __amdgpu_buffer_rsrc_t rsrc, uint32_t of) BQM_INLINE -> u32x4 {
        of = piece_ok ? of : none;
        if (a.span != 0)
            return ld_b128(rsrc, (of + piece) * 16u);
        return *(of == kNoWidePlace ? (piece_ptr)&kZeros : (piece_ptr)base + of + piece);
    };
    auto load_k = [&](u32x4 (&r)[S::kLoads], const Places &of) BQM_INLINE {
#pragma unroll
        for (int i = 0; i < S::kLoads; i++)
            r[i] = load(kh, kb_rsrc, of[i]);
    };
    auto load_v = [&](const Places &of) BQM_INLINE {
#pragma unroll
        for (int i = 0; i < S::kLoads; i++)
            vr[i] = load(vh, vb_rsrc, of[i]);
    };
    auto store_k = [&](const u32x4 (&r)[S::kLoads], char *to) BQM_INLINE {
#pragma unroll
        for (int i = 0; i < S::kLoads; i++)
            *reinterpret_cast<u32x4 *>(to + (row0 + i * S::kRowsPerLoad) * S::KS + piece * 16) = r[i];
    };
    // a tile's last resorts, each gone through again from the start: keep infinities
    // and NaN of V out of the products; and weigh less, so that no sum overflows
    bool careful = false, light = false;
    auto store_v = [&](char *to) BQM_INLINE {
#pragma unroll
        for (int i = 0; i < S::kLoads; i++) {
            if (careful)
                vr[i] = finite_only<T>(vr[i]);
            *reinterpret_cast<u32x4 *>(to + (row0 + i * S::kRowsPerLoad) * S::VS + piece * 16) = vr[i];
        }
    };

    f32x16 acc[DP / 32];
    float top, sum;  // of this lane's row; sum over its own tokens
    // log2 of what a weight at top comes to. Half precision has only 2^-25 below 1
    // (less comes out as zero) but 2^16 above: weights of up to 2^15 keep what is above
    // 2^-32 of the row's largest; a million tokens below that come to less than an
    // output's own rounding.
    float lift = __is_same(T, _Float16) ? 7.0f : 0.0f;

    // whether a row of this wave sees the tile at t0
    auto seen = [&](int t0) { return t0 < hi_last && t0 + S::TK > lo_first; };
    // The scheduler left alone puts each operand read right before its product and
    // waits; these keep kAhead reads in flight.
    constexpr int kAhead = 4;
    // operand i of the scores: the tiles of 32 tokens in turn, so that no product
    // waits for the sum of the one before it
    auto read_k = [&](const char *k, int i) BQM_INLINE {
        const char *kb = k + col * S::KS + half * 16;
        return *reinterpret_cast<const Op *>(kb + i % NT * 32 * S::KS + i / NT * 32);
    };
    auto scores = [&](Scores &s, const char *k) BQM_INLINE {
        Op f[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++)
            f[i] = read_k(k, i);
#pragma unroll
        for (int tt = 0; tt < NT; tt++)
            s[tt] = f32x16{};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NT * DP / 16; i++) {
            s[i % NT] = mfma(f[i % kAhead], qf[i / NT], s[i % NT]);
            if (i + kAhead < NT * DP / 16)
                f[i % kAhead] = read_k(k, i + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the row's maximum: masks the scores, brings the accumulators to a new base
    auto settle = [&](Scores &s, int t0) BQM_INLINE {
        if (!(t0 >= lo_last && t0 + S::TK <= hi_first)) {
#pragma unroll
            for (int tt = 0; tt < NT; tt++)
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int j = t0 + tt * 32 + (i / 4) * 8 + half * 4 + i % 4;
                    s[tt][i] = j >= lo && j < hi ? s[tt][i] : -INFINITY;
                }
        }
        float ms[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains, not one
#pragma unroll
        for (int tt = 0; tt < NT; tt++)
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                ms[i / 4] = fmaxf(fmaxf(ms[i / 4], s[tt][i]), s[tt][i + 1]);
        const float m =
            pair_max(fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]))) * a.scale_log2;
        // The weights' base follows the maximum only when that has grown by a
        // factor of 2^8: sums and weights (up to 256, the same relative rounding
        // in either type) have room for it, and most tiles pass without scaling
        // the accumulators.
        if (__any(m > top + 8.0f)) {
            const float grown = fmaxf(m, top);
            const float back = top == -INFINITY ? 0.0f : exp2_fast(top - grown);
            top = grown;
            sum *= back;
#pragma unroll
            for (int dt = 0; dt < DP / 32; dt++)
#pragma unroll
                for (int i = 0; i < 16; i++)
                    acc[dt][i] *= back;
        }
        return (top == -INFINITY ? 0.0f : top) - lift;  // the former: nothing seen yet
    };
    constexpr int kTiles = DP / 32, kChunks = 2 * NT;  // of 32 values, of 16 tokens
    auto weights = [&](f32x8 &e, const Scores &s, float base, int c, int first, int n) BQM_INLINE {
#pragma unroll
        for (int i = first; i < first + n; i++) {
            e[i] = exp2_fast(fmaf(s[c / 2][8 * (c % 2) + i], a.scale_log2, -base));
            sum += e[i];
        }
    };
    // 16 lanes read 4 tokens x 16 values; lane l gets value l of the 4
    const int v_lane = (half * 4 + (lane & 15) / 4) * S::VS + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    auto read_v = [&](const char *v, int c, int dt) BQM_INLINE {
        typedef __attribute__((address_space(3))) s16x4 *lp;
        const char *at = v + v_lane + c * 16 * S::VS + dt * 64;
        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at));
        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 8 * S::VS));
        return __builtin_bit_cast(Op, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // Weights and products, 16 tokens at a time. Between the products of 16 tokens
    // go the exponentials and the operand reads of the next 16, in this order.
    auto weigh_and_multiply = [&](const Scores &s, float base, const char *v) BQM_INLINE {
        constexpr int kShare = 8 / kTiles;
        // For an output of 32 bits what a weight's rounding leaves over is multiplied too,
        // where rows are few and memory bounds the kernel: weights of twice the bits
        // (61 ragged sequences of up to 8192 tokens 104.9 -> 105.7 us, 24 of up to 1126
        // 20.2 -> 21.1). An output of 16 bits rounds as much away itself; and with many
        // rows the products are what the kernel does, and it would do three for two.
        constexpr bool kRest = WM == 1 && sizeof(O) == 4;
        f32x8 e;
        Op f[2][kTiles];
#pragma unroll
        for (int dt = 0; dt < kTiles; dt++)
            f[0][dt] = read_v(v, 0, dt);
        __builtin_amdgcn_sched_barrier(0);
        weights(e, s, base, 0, 0, 8);
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
            // rounded to the cache's type: the matrix cores take no wider operand
            const Op p = __builtin_convertvector(e, Op);
            Op rest;
            if constexpr (kRest)
                rest = __builtin_convertvector(e - __builtin_convertvector(p, f32x8), Op);
#pragma unroll
            for (int dt = 0; dt < kTiles; dt++) {
                acc[dt] = mfma(f[c % 2][dt], p, acc[dt]);
                if constexpr (kRest)
                    acc[dt] = mfma(f[c % 2][dt], rest, acc[dt]);
                if (c + 1 < kChunks) {
                    f[(c + 1) % 2][dt] = read_v(v, c + 1, dt);
                    weights(e, s, base, c + 1, dt * kShare, kShare);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    for (;;) {
        ct = t00 + lane % S::TK;
        cpage = ct / a.page_size;
        cplace = ct % a.page_size;
#pragma unroll
        for (int dt = 0; dt < DP / 32; dt++)
            acc[dt] = f32x16{};
        top = -INFINITY;
        sum = 0.0f;
        look_up();
        if constexpr (kHalves) {
            // Step n of a half: at its products, S(n + 1) from K(n + 1) and the
            // sums from V(n) and the weights n; then, while the other half is at
            // its products, the weights n + 1 and its share of the next tiles to
            // LDS. The first half is at products n in phase 2n, the second in phase
            // 2n + 1, so K(n + 2) and V(n + 1) may be stored in phases 2n (by the
            // second half, between its steps n - 1 and n) and 2n + 1 (by the first):
            // what they replace was last read in phase 2n - 1.
            const bool second = wm >= 4;
            Places of_k, of_v;
            {  // K(0), K(1) and V(0) in one round of loads
                const int page0 = page_id, place0 = place;
                look_up();
                const int page1 = page_id, place1 = place;
                look_up();
                const int page2 = page_id, place2 = place;
                page_id = page0, place = place0;
                spread(of_v, place_of());
                page_id = page1, place = place1;
                spread(of_k, place_of());
                page_id = page2, place = place2;
            }
            u32x4 k0[S::kLoads];
            load_k(k0, of_v);
            load_k(kr, of_k);
            load_v(of_v);
            store_k(k0, k_of(0));
            store_k(kr, k_of(1));
            store_v(v_of(0));
#pragma unroll
            for (int i = 0; i < S::kLoads; i++)
                of_v[i] = of_k[i];
            spread(of_k, place_of());
            look_up();
            load_v(of_v);  // V(1), K(2)
            load_k(kr, of_k);
            __syncthreads();
            Scores s;
            Op p[kChunks];
            auto soften = [&](int n) BQM_INLINE {  // the weights n
                const int t0 = t00 + n * S::TK;
                if (!seen(t0)) {
#pragma unroll
                    for (int c = 0; c < kChunks; c++)
                        p[c] = Op{};
                    return;
                }
                const float base = settle(s, t0);
#pragma unroll
                for (int c = 0; c < kChunks; c++) {
                    f32x8 e;
                    weights(e, s, base, c, 0, 8);
                    // rounded to the cache's type: the matrix cores take no wider operand
                    p[c] = __builtin_convertvector(e, Op);
                }
            };
            // K(n + 2) and V(n + 1) to LDS, the loads of the tiles after them, and
            // the weights m
            auto stage_and_soften = [&](int n, int m) BQM_INLINE {
                store_k(kr, k_of(n));
                store_v(v_of(n + 1));
#pragma unroll
                for (int i = 0; i < S::kLoads; i++)
                    of_v[i] = of_k[i];
                spread(of_k, place_of());
                look_up();
                load_v(of_v);
                load_k(kr, of_k);
                soften(m);
            };
            scores(s, k_of(0));
            if (!second)
                soften(0);
            __syncthreads();
            if (second) {
                stage_and_soften(0, 0);
                __syncthreads();
            }
            for (int n = 0; n < iters; n++) {
                const int t0 = t00 + n * S::TK;
                if (seen(t0) || seen(t0 + S::TK)) {
                    // S(n + 1), then the products with V(n), reads kAhead of them
                    constexpr int kScores = NT * DP / 16, kAll = kScores + kChunks * kTiles;
                    const char *k = k_of(n + 1), *v = v_of(n);
                    auto read = [&](int i) {
                        return i < kScores ? read_k(k, i)
                                           : read_v(v, (i - kScores) / kTiles, (i - kScores) % kTiles);
                    };
                    Op f[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; i++)
                        f[i] = read(i);
#pragma unroll
                    for (int tt = 0; tt < NT; tt++)
                        s[tt] = f32x16{};
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < kAll; i++) {
                        if (i < kScores) {
                            s[i % NT] = mfma(f[i % kAhead], qf[i / NT], s[i % NT]);
                        } else {
                            const int c = (i - kScores) / kTiles, dt = (i - kScores) % kTiles;
                            acc[dt] = mfma(f[i % kAhead], p[c], acc[dt]);
                        }
                        if (i + kAhead < kAll)
                            f[i % kAhead] = read(i + kAhead);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                __syncthreads();
                stage_and_soften(second ? n + 1 : n, n + 1);
                __syncthreads();
            }
            if (!second)
                __syncthreads();
        } else {
            auto load_both = [&]() BQM_INLINE {
                Places of;
                spread(of, place_of());
                look_up();
                load_k(kr, of);
                load_v(of);
            };
            auto store_both = [&](int n) BQM_INLINE {
                store_k(kr, k_of(n));
                store_v(v_of(n));
            };
            auto compute = [&](int n) BQM_INLINE {
                const int t0 = t00 + n * WK * S::TK;
                if (!seen(t0))
                    return;
                Scores s;
                scores(s, k_of(n));
                const float base = settle(s, t0);
                weigh_and_multiply(s, base, v_of(n));
            };
            load_both();
            if constexpr (S::kBufs == 1) {
                // each wave has its own tile: no barrier, the next tile loads into
                // registers while this one is used
                for (int n = 0; n < iters; n++) {
                    store_both(n);
                    load_both();
                    compute(n);
                }
            } else {
                store_both(0);
                load_both();
                __syncthreads();
                for (int n = 0; n < iters; n++) {
                    store_both(n + 1);
                    load_both();
                    compute(n);
                    __syncthreads();
                }
            }
        }
        // A weight of zero that met an infinity or NaN in a value its row does not
        // see leaves NaN: then all again with those values as zeros, and rows that
        // do see them get their due at the end. Sums of finite values above 2^120
        // are taken again too, with weights so low that all of them together come to
        // less than one: neither they nor the sum of four waves or many parts can
        // then overflow, as sums of values near bfloat16's largest, 2^128, would at
        // weights of up to 2^8. (Lower weights are lost below 2^-126, which is why
        // they are not taken so from the start.) Rows of NaN sums are NaN throughout.
        const float all = pair_sum(sum);
        bool odd = false;
#pragma unroll
        for (int dt = 0; dt < DP / 32; dt++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                odd |= !(fabsf(acc[dt][i]) < 0x1p120f);
        if (light || !__syncthreads_or(odd && all == all)) {
            sum = all;
            break;
        }
        light = careful;
        careful = true;
        if (light) {  // tokens < 2^(32 - clz), weights <= 2^(8 + lift)
            const float low = (float)(__builtin_clz(max(c1 - c0, 1)) - 40);
            lift = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(low)));
        }
    }

    const int64_t part_row = (int64_t)split * a.total_q * a.n_q_heads;
    // What the careful products left out: infinities and NaN that the rows see
    // (their weights are above zero, whatever they round to) are the output in
    // their places.
    auto left_out = [&](bool stores, int first, int step) {
        auto value_of = [&](int j) -> const T * {  // of token j
            const int page = j < c1 ? table[j / a.page_size] : -1;
            if ((uint32_t)page >= (uint32_t)a.n_pages)
                return nullptr;
            return reinterpret_cast<const T *>(a.v) +
                   8 * ((int64_t)page * a.c_page + (int64_t)(j % a.page_size) * a.c_token +
                        (int64_t)head * a.c_head);
        };
        __threadfence_block();  // the rows' stores come first
#pragma unroll 1
        for (int d = first * 32 + half; d < a.dim; d += d % 32 < 30 ? 2 : 32 * step - 30) {
            float o = 0.0f;
#pragma unroll 1
            for (int j0 = c0; j0 < c1; j0 += 64) {
                const T *v = value_of(j0 + lane);
                const int d_even = d - half;
                const bool bad = v && !(fabsf((float)v[d_even]) < INFINITY &&
                                        fabsf((float)v[d_even + 1]) < INFINITY);
#pragma unroll 1
                for (uint64_t bads = __ballot(bad); bads; bads &= bads - 1) {
                    const int j = j0 + __builtin_ctzll(bads);
                    const float x = (float)value_of(j)[d];
                    if (j >= lo && j < hi && !(fabsf(x) < INFINITY))
                        o += x;
                }
            }
            if (stores && !(fabsf(o) < INFINITY)) {
                if (parts > 1)
                    a.part[(part_row + out_row) * a.dim + d] = o;
                else
                    static_cast<O *>(a.out)[out_row * a.dim + d] = (O)o;
            }
        }
    };
    // The output's 32-value tiles first, first + step, .. (o(dt)):
    // final, or this part's share with its maximum m and sum l.
    auto store_out = [&](auto o, int first, int step, float m, float l) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const bool stores = col < t.rows - row_first;
#pragma unroll
        for (int dt = first; dt < DP / 32; dt += step) {
            const f32x16 w = o(dt);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const f32x4 v = {w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
                const int d = dt * 32 + c * 8 + half * 4;
                if (stores && d < a.dim) {
                    if (parts > 1)
                        store4(a.part + (part_row + out_row) * a.dim + d, v);
                    else
                        store4(static_cast<O *>(a.out) + out_row * a.dim + d, v * inv);
                }
            }
        }
        if (stores && parts > 1 && first == 0 && half == 0)
            a.part_ml[part_row + out_row] = make_float2(m - lift, l);
        // the lanes share out the tokens, so all of them take part, those too whose row
        // a sum of NaN has made NaN already
        if (careful)
            left_out(stores && l == l, first, step);
    };

    if constexpr (WK == 1) {
        store_out([&](int dt) { return acc[dt]; }, 0, 1, top, sum);
    } else {
        // join the groups: every wave brings its sums to the common maximum, and
        // each 32-value tile is added up by one of them
        static_assert(WM == 1, "the join is written for groups of one wave");
        float *ml = reinterpret_cast<float *>(lds + WK * (DP / 32) * 4096);
        float *os = reinterpret_cast<float *>(lds);
        __syncthreads();
        if (half == 0)
            ml[wk * 32 + col] = top;
        __syncthreads();
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WK; w++)
            m = fmaxf(m, ml[w * 32 + col]);
        const float f = top == -INFINITY ? (sum == sum ? 0.0f : 1.0f) : exp2_fast(top - m);
        float *ls = ml + WK * 32;
        if (half == 0)
            ls[wk * 32 + col] = sum * f;
#pragma unroll
        for (int dt = 0; dt < DP / 32; dt++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                os[((wk * (DP / 32) + dt) * 16 + i) * 64 + lane] = acc[dt][i] * f;
        __syncthreads();
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < WK; w++)
            l += ls[w * 32 + col];
        store_out(
            [&](int dt) {
                f32x16 o = {};
#pragma unroll
                for (int w = 0; w < WK; w++)
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        o[i] += os[((w * (DP / 32) + dt) * 16 + i) * 64 + lane];
                return o;
            },
            wk, WK, m, l);
    }
}

// Joins the parts of rows whose tokens were cut. WAVES waves share a row and
// take every WAVES-th part, several parts' loads in flight in each: four for the
// many parts of a long sequence (64 rows of 62 parts 7.8 us, of 32 parts 5.6; one
// wave a row took 89 for 62), one where rows are many and parts few (2048 rows of up to 8: 5.6 us; a
// workgroup each 7.3). Latency bounds both: three loads that follow each other.
constexpr int kMostParts = 1024;
constexpr int kFewParts = 16;

template <class O, int M, int WAVES>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a)
{
    constexpr int kRows = 4 / WAVES;  // of a workgroup
    __shared__ float weights[kRows][WAVES == 1 ? kFewParts : kMostParts];
    __shared__ float shares[4][256], sums[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slot = wave / WAVES, part0 = wave % WAVES;
    const int64_t rows = a.total_q * a.n_q_heads, row = (int64_t)blockIdx.x * kRows + slot;
    int parts = 1;
    if (row < rows) {
        const int64_t tq = row / a.n_q_heads;
        const int h = (int)(row - tq * a.n_q_heads);
        Tile t;
        load_sequence(a, find_sequence(a, tq, [](int start, int) { return (int64_t)start; }), t);
        if (tq >= t.q0 && tq < t.q0 + t.q_len) {
            t.tile = (int)((tq - t.q0) * a.group + h % a.group) / M;
            load_range<M>(a, t);
            parts = parts_of(a, t);
        }
    }
    if (WAVES > 1 ? parts == 1 : __syncthreads_and(parts == 1))
        return;  // written whole; the row is the workgroup's, or none of its rows is cut
    // every wave finds its row's maximum; the parts' weights go to LDS
    const float2 *mls = a.part_ml + row;
    float m = -INFINITY, l = 0.0f;
    if (parts > 1)
        for (int p = lane; p < parts; p += 64)
            m = fmaxf(m, mls[p * rows].x);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        m = fmaxf(m, __shfl_xor(m, d, 64));
    const float base = m == -INFINITY ? 0.0f : m;
    float *weight = weights[slot];
    if (parts > 1)
        for (int p = part0 * 64 + lane; p < parts; p += 64 * WAVES) {
            const float2 ml = mls[p * rows];
            const float f =
                ml.x == -INFINITY ? (ml.y == ml.y ? 0.0f : 1.0f) : exp2_fast(ml.x - base);
            weight[p] = f;
            l += ml.y * f;
        }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        l += __shfl_xor(l, d, 64);
    if (lane == 0)
        sums[wave] = l;
    __syncthreads();
    if constexpr (WAVES > 1)
        l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    f32x4 o = {};
    if (parts > 1 && lane * 4 < a.dim) {
        const float *src = a.part + row * a.dim + lane * 4;
#pragma unroll 4
        for (int p = part0; p < parts; p += WAVES) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(src + p * rows * a.dim);
            // an infinity stays one where its part's weight has come out as zero
            const float w = weight[p] * inv;  // before the sum: shares of a mean cannot overflow
#pragma unroll
            for (int i = 0; i < 4; i++)
                o[i] += fabsf(v[i]) < INFINITY ? v[i] * w : v[i];
        }
    }
    if constexpr (WAVES == 1) {
        if (parts > 1 && lane * 4 < a.dim)
            store4(static_cast<O *>(a.out) + row * a.dim + lane * 4, o);
    } else {
        static_assert(WAVES == 4, "the workgroup's waves share one row");
        *reinterpret_cast<f32x4 *>(&shares[wave][lane * 4]) = o;
        __syncthreads();
        const int d = threadIdx.x;
        if (d < a.dim) {
            const float v = (shares[0][d] + shares[1][d]) + (shares[2][d] + shares[3][d]);
            static_cast<O *>(a.out)[row * a.dim + d] = (O)v;
        }
    }
}

// How a call is launched: which kernel, and into how many parts the tokens of a
// tile are cut so that the card is full when there are few rows.
struct Plan {
    int m;              // rows a workgroup: 32 (its four waves on tokens), 128 or 256
    int tiles, n_splits, chunk;
};

constexpr int kFewRows = 32;
constexpr int64_t kLeastSaved = 512, kLeastSavedOf64 = 832, kLeastSavedFew = 256;
constexpr int64_t kRaggedWorkgroups = 128;   // 16 of 100 to 8000 tokens: 30 us, uncut by this 37
constexpr int64_t kManyTiles = 512;          // of 256 rows: two a compute unit
constexpr int64_t kManyTokens = 2048;
constexpr int64_t kMostWorkgroups = 8192;    // most of them empty, where lengths differ
constexpr int kLeastChunk = 256, kRaggedChunk = 1024;

// Workgroups, parts counted, that a launch is cut into.
// Tiles of 32 rows: no more than run at once, two a compute unit, since what does not takes
// another round (24 tokens over 1126, heads of 128, 192 tiles: 33 us in two parts, 40
// in three; 12 over 3000: 41 us in five, 45 in nine), and one part where several would
// spare no more than kLeastSavedFew tokens (64 over 300: 22 us in one, 33 in two).
// Tiles of 128 rows: the nearest number of parts is taken, and one where several would spare
// a workgroup no more than kLeastSaved tokens: their shares' way costs as much (28 heads
// of 64 over 4, 17 x 72 tokens with a window of 1024: 49 us in two parts, 32 in one;
// a prompt of 1024, heads of 128: 41 and 33). Heads of 64 run three workgroups a
// compute unit (17 x 36 tokens over 4096: 70 us in one part, 55 in three; 17 x 108,
// 408 tiles: 94 in one, 130 in two). Heads of 128 run two; where a sequence's tiles are
// one or two, its keys and values are hardly read again, memory bounds them and more
// parts only add to that (8 x 64 tokens over 4096: 76 us in three parts, 88 in four;
// 32 x 32 over 4096: 153 in one, 186 in two), but not where many share them (512 tokens
// over 8192: 98 us in four parts, 113 in three). Heads of 256 run one, in rounds (4 x 128
// tokens over 4096: 103 us in seven parts, 110 in six, 127 in eight).
int64_t wanted_tiles(int head_dim, int64_t of_one, bool few)
{
    if (few)
        return 512;
    if (head_dim <= 64)
        return 576;
    if (head_dim > 128)
        return 432;
    return of_one <= 2 ? 352 : 512;
}

// window: 0 if none bounds what a tile's rows see between them (rows that see later
// tokens reach to the sequence's end)
Plan plan_of(const bqm_kv_cache *c, const bqm_kv_batch *b, int n_q_heads, int window)
{
    const int64_t group = n_q_heads / c->n_heads;
    Plan p;
    const int64_t rows = b->total_q * group;
    const bool few = std::min<int64_t>(b->max_q, b->total_q) * group <= kFewRows;
    int64_t seen = std::min<int64_t>(b->max_kv, (int64_t)b->max_pages * c->page_size);
    if (window > 0)
        seen = std::min<int64_t>(seen, window);
    // 256 rows in two halves: heads of 65 to 128 values, enough tiles for two a
    // compute unit, and enough tokens for a workgroup's start and end, which nothing
    // covers, to be small (32 heads of 128, prompts of 4096 and 8192 tokens: 156 and
    // 571 us, with 128 rows 176 and 608; of 2048, half the tiles: 86 and 62; four of
    // 2048 with a window of 512: 118 and 113; heads of 64, 8192 tokens: 399 and 336).
    const bool many = c->head_dim > 64 && c->head_dim <= 128 &&
                      rows / 256 * c->n_heads >= kManyTiles && seen >= kManyTokens;
    const int m = p.m = few ? 32 : many ? 256 : 128;
    p.tiles = (int)(rows / m + b->n_seqs);
    // the most tokens a tile's rows see between them
    int64_t room = std::min<int64_t>(b->max_kv, (int64_t)b->max_pages * c->page_size);
    if (window > 0)
        room = std::min<int64_t>(room, (int64_t)window + m / group + 1);
    const int64_t workgroups = (int64_t)p.tiles * c->n_heads;
    // parts that fill the card, if every sequence had max_q rows and max_kv tokens
    // tiles of one sequence, and of all
    const int64_t of_one = std::max<int64_t>(
        1, (std::min<int64_t>(b->max_q, b->total_q) * group + m - 1) / m);
    const int64_t most_tiles = std::min<int64_t>(p.tiles, b->n_seqs * of_one) * c->n_heads;
    const int64_t wanted = wanted_tiles(c->head_dim, of_one, few);
    const int64_t parts = std::max<int64_t>(1, (wanted + (few ? 0 : most_tiles / 2)) / most_tiles);
    int64_t chunk = (room + parts - 1) / parts;
    const int64_t least = few ? kLeastSavedFew : c->head_dim <= 64 ? kLeastSavedOf64 : kLeastSaved;
    if (m == 256 || room - chunk <= least)
        chunk = room;
    chunk = std::max<int64_t>(kLeastChunk, chunk);
    // Many sequences of few rows: cut the long among the short ones too (64 of 33 to
    // 8192 tokens: 104 us at 1024 tokens a part, 110 at 512, 107 at 2048). Few
    // sequences are cut enough already (2 of 131071: 184 us at 4096, 188 at 2048, 197 at 1024).
    if (few && workgroups >= kRaggedWorkgroups)
        chunk = std::min(chunk,
                         std::max<int64_t>(kRaggedChunk, room * workgroups / kMostWorkgroups));
    // no more parts than the workspace holds, whose size does not know the window
    const int64_t most =
        window > 0 ? plan_of(c, b, n_q_heads, 0).n_splits : (int64_t)kMostParts;
    chunk = std::max(chunk, (room + most - 1) / most);
    p.chunk = (int)((chunk + 127) / 128 * 128);
    p.n_splits = (int)std::max<int64_t>(1, (room + p.chunk - 1) / p.chunk);
    return p;
}

template <class T, class O, int DP, int WM, int WK, int NT, int WAVES>
int launch_shape(const AttnArgs &a, hipStream_t stream)
{
    typedef Shape<DP, WM, WK, NT> S;
    auto kernel = attention_kernel<T, O, DP, WM, WK, NT, WAVES>;
    allow_dynamic_lds(reinterpret_cast<const void *>(kernel), S::kLds);
    const int64_t grid = (int64_t)a.tiles * a.n_splits * a.n_heads;
    if (grid * S::kThreads >= 1ll << 32)
        return BQM_ERR_SHAPE;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(S::kThreads), S::kLds, stream, a);
    const int64_t rows = a.total_q * a.n_q_heads;
    if constexpr (S::M < 256) {
        if (a.n_splits > kFewParts)
            hipLaunchKernelGGL((attention_join_kernel<O, S::M, 4>), dim3((unsigned)rows), dim3(256),
                               0, stream, a);
        else if (a.n_splits > 1)
            hipLaunchKernelGGL((attention_join_kernel<O, S::M, 1>), dim3((unsigned)((rows + 3) / 4)),
                               dim3(256), 0, stream, a);
    }
    return check_launch();
}

template <class T, class O, int DP>
int launch_rows(const AttnArgs &a, int m, hipStream_t stream)
{
    constexpr int kWaves = DP > 128 ? 1 : DP > 64 ? 2 : 3;  // a SIMD's, by the registers
    if (m == 32)
        return launch_shape<T, O, DP, 1, 4, 1, kWaves>(a, stream);
    if constexpr (DP == 128)
        if (m == 256)
            return launch_shape<T, O, DP, 8, 1, 2, 2>(a, stream);
    return launch_shape<T, O, DP, 4, 1, 2, kWaves>(a, stream);
}

template <class T, class O>
int launch_types(const AttnArgs &a, int m, hipStream_t stream)
{
    if (a.dim <= 64)
        return launch_rows<T, O, 64>(a, m, stream);
    if (a.dim <= 128)
        return launch_rows<T, O, 128>(a, m, stream);
    return launch_rows<T, O, 256>(a, m, stream);
}

}  // namespace

size_t attention_workspace(const bqm_kv_cache *c, const bqm_kv_batch *b, int n_q_heads)
{
    if (b->total_q == 0)
        return 0;
    const Plan p = plan_of(c, b, n_q_heads, 0);
    if (p.n_splits == 1)
        return 0;
    const size_t rows = (size_t)p.n_splits * b->total_q * n_q_heads;
    return (rows * (4 * (size_t)c->head_dim + 8) + 255) / 256 * 256;
}

int launch_paged_attention(const void *q, int64_t q_token, int64_t q_head, const bqm_kv_cache *c,
                           const bqm_kv_batch *b, void *out, int n_q_heads, float scale,
                           bool causal, int window, int out_dtype, void *workspace,
                           hipStream_t stream)
{
    const Plan p = plan_of(c, b, n_q_heads, causal ? window : 0);
    AttnArgs a = {};
    a.q = q;
    a.k = static_cast<const u32x4 *>(c->k);
    a.v = static_cast<const u32x4 *>(c->v);
    a.out = out;
    a.pages = b->table;
    a.kv_lens = b->kv_lens;
    a.q_starts = b->q_starts;
    a.q_token = q_token;
    a.q_head = q_head;
    a.pages_stride = b->table_stride;
    a.total_q = b->total_q;
    a.c_page = (uint32_t)(c->page_stride / 8);
    a.c_token = (uint32_t)(c->token_stride / 8);
    a.c_head = (uint32_t)(c->head_stride / 8);
    const uint64_t span = ((uint64_t)(c->n_pages - 1) * a.c_page +
                           (uint64_t)(c->page_size - 1) * a.c_token + c->head_dim / 8) * 16;
    a.span = span <= 16ull * kNoPlace ? (uint32_t)span : 0;
    a.n_pages = (int)c->n_pages;
    a.n_seqs = b->n_seqs;
    a.max_pages = b->max_pages;
    a.page_size = c->page_size;
    a.max_kv = b->max_kv;
    a.n_q_heads = n_q_heads;
    a.n_heads = c->n_heads;
    a.group = n_q_heads / c->n_heads;
    a.dim = c->head_dim;
    a.tiles = p.tiles;
    a.n_splits = p.n_splits;
    a.chunk = p.chunk;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.causal = causal;
    a.window = window;
    a.part = static_cast<float *>(workspace);
    if (p.n_splits > 1)
        a.part_ml = reinterpret_cast<float2 *>(
            a.part + (size_t)p.n_splits * b->total_q * n_q_heads * c->head_dim);
    if (c->dtype == BQM_DTYPE_F16)
        return out_dtype == BQM_DTYPE_F32
                   ? launch_types<_Float16, float>(a, p.m, stream)
                   : launch_types<_Float16, _Float16>(a, p.m, stream);
    return out_dtype == BQM_DTYPE_F32 ? launch_types<__bf16, float>(a, p.m, stream)
                                      : launch_types<__bf16, __bf16>(a, p.m, stream);
}

}  // namespace bqm
