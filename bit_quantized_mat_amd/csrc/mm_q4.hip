// mm_q4.hip -- product of a 4-bit matrix (layout in include/bqm.h) and Q8_1
// activation columns:
//   y[t][n] = sum_j scale * d_a[t][j] * sum_{i < 32} (code - zero) * q[t][32j + i].
//
// The inner sums are exact whole numbers. A code's nibble kept in the high half of
// its byte is 16 times the code as int8, so the low halves need a shift and a mask
// and the high ones a mask; the 16 goes into d_a.
//
// Three kernels: one or two columns go without the matrix cores, bound by reading the matrix;
// columns that fit in LDS, at most 32, stay there while waves stream rows; more go by tiles,
// where vector and matrix instructions and waits add up. Each keeps the header's bound, 1e-5 of
// the terms' sum, by the number of roundings that a term goes through. Figures are of one MI355X.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

struct Q4Args {
    bqm_q4_matrix m;
    const uint8_t *a;
    float *y;
    int64_t T;
    int nb;     // runs of 32 in a row
    int shift;  // log2(group / 32)
};

constexpr int kStageRuns = 128;  // runs of a column staged at once

// Columns 0 .. TC - 1 of runs b0 .. b0 + n - 1, as two planes of 16 bytes a run
// (a lane reads each with one load, neighbours next to each other), d / 16 and sums.
template <int TC>
struct Stage {
    uint4 lo[TC][kStageRuns], hi[TC][kStageRuns];
    float d[TC][kStageRuns];
    int sum[TC][kStageRuns];
};

template <int TC, bool Z>
__device__ __forceinline__ void stage_columns(Stage<TC> &s, const Q4Args &g, int b0, int n)
{
    for (int i = threadIdx.x; i < TC * kStageRuns; i += 256) {
        const int t = i / kStageRuns, b = i % kStageRuns;
        if (b >= n)
            continue;
        const int64_t col = t < g.T ? t : g.T - 1;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(
            g.a + (col * g.nb + b0 + b) * kQ81BlockBytes);
        uint32_t q[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            q[k] = p[k];
        s.lo[t][b] = make_uint4(q[0], q[1], q[2], q[3]);
        s.hi[t][b] = make_uint4(q[4], q[5], q[6], q[7]);
        s.d[t][b] = f16_bits_to_f32(p[8] & 0xffffu) * 0.0625f;
        if constexpr (Z) {
            int sum = 0;
#pragma unroll
            for (int k = 0; k < 8; k++)
                sum = sdot4(q[k], 0x01010101u, sum);
            s.sum[t][b] = 16 * sum;
        }
    }
}

// A wave has R rows at a time of each of its 64 >> lr lane groups; lanes of a group take
// the row's runs in turn. Rows are read once, 16 bytes a lane, R loads on their way. 100003 x
// 4096 and one column: 41.6 us, 5.2 TB/s (a large copy: 5.1); 4096 x 4096 4.5, latency. Two
// columns 48; four took 67 to 75 and eight 120, where the next kernel takes 52.
//
// A term goes through a rounding of its own, one a run that follows in its lane's sum and six where
// lanes are added; the header's 1e-5 are 167. LONG: rows of which a lane has more runs than that
// have a sum of each kSumRuns, 128 of a lane, added up one after another (four at most).
constexpr int kSumRuns = 64 * kStageRuns;

template <int TC, int R, bool Z, bool LONG>
__global__ __launch_bounds__(256) void q4_dot_kernel(const Q4Args g, int lr)
{
    __shared__ Stage<TC> s;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int per = 64 >> lr;  // rows side by side
    const int64_t first = (block_of_grid() * 4 + wave) * (per * R) + (lane >> lr);
    float acc[R][TC] = {}, before[R][TC];
    for (int b0 = 0; b0 < g.nb; b0 += kStageRuns) {
        const int n = g.nb - b0 < kStageRuns ? g.nb - b0 : kStageRuns;
        if constexpr (LONG) {
            if (b0 % kSumRuns == 0) {
#pragma unroll
                for (int i = 0; i < R * TC; i++) {
                    before[i / TC][i % TC] =
                        b0 ? before[i / TC][i % TC] + acc[i / TC][i % TC] : 0.0f;
                    acc[i / TC][i % TC] = 0.0f;
                }
            }
        }
        if (b0)
            __syncthreads();
        stage_columns<TC, Z>(s, g, b0, n);
        __syncthreads();
        for (int b = lane & ((1 << lr) - 1); b < n; b += 1 << lr) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                int64_t row = first + r * per;
                row = row < g.m.N ? row : g.m.N - 1;
                const uint4 c = static_cast<const uint4 *>(g.m.codes)[row * g.nb + b0 + b];
                const int64_t at = row * (g.nb >> g.shift) + ((b0 + b) >> g.shift);
                const float scale = f16_bits_to_f32(static_cast<const uint16_t *>(g.m.scales)[at]);
                const int zero = Z ? g.m.zeros[at] : 0;
                const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int t = 0; t < TC; t++) {
                    const uint4 l = s.lo[t][b], h = s.hi[t][b];
                    const uint32_t ls[4] = {l.x, l.y, l.z, l.w}, hs[4] = {h.x, h.y, h.z, h.w};
                    int sum = 0;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        sum = sdot4((cs[k] << 4) & 0xf0f0f0f0u, ls[k], sum);
                        sum = sdot4(cs[k] & 0xf0f0f0f0u, hs[k], sum);
                    }
                    if constexpr (Z)
                        sum -= zero * s.sum[t][b];
                    acc[r][t] = fmaf(scale, s.d[t][b] * (float)sum, acc[r][t]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int64_t row = first + r * per;
#pragma unroll
        for (int t = 0; t < TC; t++) {
            const float v = row_sum(LONG ? before[r][t] + acc[r][t] : acc[r][t], lr);
            if ((lane & ((1 << lr) - 1)) == 0 && row < g.m.N && t < g.T)
                g.y[t * g.m.N + row] = v;
        }
    }
}

template <int TC, int R>
int launch_dot(const Q4Args &g, hipStream_t stream)
{
    int lr = 0;
    while (lr < 6 && (1 << lr) < g.nb)
        lr++;
    const int rows = 4 * R * (64 >> lr);
    const dim3 grid = grid_of((g.m.N + rows - 1) / rows);
    auto run = [&](auto *kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, g, lr);
        return check_launch();
    };
    if (g.nb > kSumRuns)
        return g.m.zeros ? run(q4_dot_kernel<TC, R, true, true>)
                         : run(q4_dot_kernel<TC, R, false, true>);
    return g.m.zeros ? run(q4_dot_kernel<TC, R, true, false>)
                     : run(q4_dot_kernel<TC, R, false, false>);
}

// ---- many columns: the matrix cores ------------------------------------------------
//
// Codes less zeros (-15 .. 15) and q (-127 .. 127) are exact in fp16, and sums over a run
// of 32 are exact in fp32, so a 16 x 16 tile of a run is one 16x16x32 product whose result
// needs one fma by d_a, and one by the scale at the end of a group. Eight codes become
// fp16 in nine instructions: a nibble under the exponent of 1024 is 1024 + nibble.
//
// A lane of group h (lane / 16) takes dword h of a row's run: the values 4h + {0, 2},
// 16 + 4h + {0, 2}, 4h + {1, 3}, 16 + 4h + {1, 3}. The columns are laid out once a call, in
// the order in which lanes read them: an operand's 64 lanes x 16 bytes in a row.

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileCols = 32;    // columns of a tile
constexpr int kChunkRuns = 4;    // runs between two barriers
constexpr int kOperand = 2048;   // bytes of one tile's run: two operands

// Workspace: operands [column tile][run][half of the columns][64][16 bytes], then d [column tile][run][32]
// fp32; runs padded to whole chunks, columns to whole tiles, with zeros.
// Where there are few tiles, the runs are cut into parts, whose sums [part][T][N] come after.
struct Laid {
    char *ops;
    float *d, *sums;
    int runs, tiles, parts;
    int stretch;  // chunks that go into one sum
};

// A term's roundings, 2^-24 each, have to stay below the 167 that are the header's 1e-5: those of
// its group (1 << SH), one a group that follows in its sum, one a sum that is added to it. So a
// part is cut into the fewest stretches that keep within that, summed one after another in y; one
// sum takes 164 groups of 32 (5248 values), 162 of 128 (20736). Returns a stretch's chunks, 0 if no
// number of stretches does.
constexpr int kMostRoundings = 166;
int stretch_of(int64_t chunks, int parts, int shift)
{
    const int64_t part = (chunks + parts - 1) / parts;
    for (int n = 1; n <= kMostRoundings; n++) {
        const int64_t each = (part + n - 1) / n;
        if ((1 << shift) + each * kChunkRuns / (1 << shift) + n - 1 + parts - 1 <= kMostRoundings)
            return (int)each;
    }
    return 0;
}

// Parts for N rows and T columns: as many as fill the device's 512 places, of four chunks
// (512 values) at least. 4096 x 4096 and 64 columns: 22 us in 16 parts, 41 in one; two parts
// cost more than they give (14336 x 4096, 256 columns: 76 us in two, 70 in one). The longest
// rows are cut in any case (2^20 values in groups of 32: six parts).
int parts_of(int64_t N, int64_t T, int64_t nb, int shift)
{
    const int64_t tiles = (T + kTileCols - 1) / kTileCols;
    const int64_t groups = (N + 127) / 128 * (tiles <= 2 ? 1 : (tiles + 3) / 4);
    const int64_t chunks = (nb + kChunkRuns - 1) / kChunkRuns;
    int parts = (int)std::min<int64_t>({512 / groups, chunks / 4, 16});
    parts = parts > 2 ? parts : 1;
    while (!stretch_of(chunks, parts, shift))
        parts++;
    return parts;
}

size_t padded_runs(int64_t nb) { return (nb + kChunkRuns - 1) / kChunkRuns * kChunkRuns; }

size_t laid_out_bytes(int64_t N, int64_t T, int64_t nb, int shift)
{
    const int64_t parts = parts_of(N, T, nb, shift);
    return (size_t)((T + kTileCols - 1) / kTileCols) * padded_runs(nb) *
               (kOperand + kTileCols * 4) +
           (parts > 1 ? (size_t)parts * T * N * 4 : 0);
}

Laid laid_out(void *workspace, int64_t N, int64_t T, int nb, int shift)
{
    Laid l;
    l.runs = (int)padded_runs(nb);
    l.tiles = (int)((T + kTileCols - 1) / kTileCols);
    l.parts = parts_of(N, T, nb, shift);
    l.stretch = stretch_of(l.runs / kChunkRuns, l.parts, shift);
    l.ops = static_cast<char *>(workspace);
    l.d = reinterpret_cast<float *>(l.ops + (size_t)l.tiles * l.runs * kOperand);
    l.sums = l.d + (size_t)l.tiles * l.runs * kTileCols;
    return l;
}

__device__ __forceinline__ uint32_t as_u32(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x2 as_f16x2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

// Four q as fp16: bytes 0 and 2, bytes 1 and 3.
__device__ __forceinline__ void halves_of(uint32_t q, uint32_t &even, uint32_t &odd)
{
    const uint32_t u = q ^ 0x80808080u;  // q + 128
    const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    even = as_u32(as_f16x2(__builtin_amdgcn_perm(0x64646464u, u, 0x04020400u)) - bias);
    odd = as_u32(as_f16x2(__builtin_amdgcn_perm(0x64646464u, u, 0x04030401u)) - bias);
}

// A thread a column's run.
__global__ __launch_bounds__(256) void q4_columns_kernel(const uint8_t *__restrict__ a, Laid l,
                                                         int64_t T, int nb)
{
    const int c = threadIdx.x & 31, run = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int tile = blockIdx.y;
    const int64_t col = (int64_t)tile * kTileCols + c;
    if (run >= l.runs)
        return;
    uint32_t q[8] = {};
    float d = 0.0f;
    if (col < T && run < nb) {
        const uint32_t *p =
            reinterpret_cast<const uint32_t *>(a + (col * nb + run) * kQ81BlockBytes);
#pragma unroll
        for (int k = 0; k < 8; k++)
            q[k] = p[k];
        d = f16_bits_to_f32(p[8] & 0xffffu);
    }
    char *to = l.ops + ((size_t)tile * l.runs + run) * kOperand + (c >> 4) * 1024 + (c & 15) * 16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint4 v;
        halves_of(q[j], v.x, v.z);
        halves_of(q[j + 4], v.y, v.w);
        *reinterpret_cast<uint4 *>(to + j * 256) = v;
    }
    l.d[((size_t)tile * l.runs + run) * kTileCols + c] = d;
}

// Bits of w turned by c where mask is set, c elsewhere: the nibbles of a mask, plus 8,
// under an exponent.
__device__ __forceinline__ f16x2 under(uint32_t w, uint32_t mask, uint32_t c)
{
    return as_f16x2(__builtin_amdgcn_bitop3_b32(w, mask, c, 0x6a));
}

// A dword of codes as an operand; low, high: minus (1032 + zero) and (72 + zero), twice.
// (High nibbles stand for 16 times themselves; nothing is rounded.)
__device__ __forceinline__ f16x8 codes_of(uint32_t w, f16x2 low, f16x2 high)
{
    const f16x2 part = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t v = w >> 8;
    const f16x2 a = under(w, 0x000f000fu, 0x64086408u) + low;
    const f16x2 b =
        __builtin_elementwise_fma(under(w, 0x00f000f0u, 0x64806480u), part, high);
    const f16x2 c = under(v, 0x000f000fu, 0x64086408u) + low;
    const f16x2 d =
        __builtin_elementwise_fma(under(v, 0x00f000f0u, 0x64806480u), part, high);
    return {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// No unit is full: scaling each run's result costs more than the product, and both more or less
// add up. Of a 14336 x 4096 product of 2000 columns' 340 to 350 us (690 TFLOP/s; a large fp16
// library product 1244) vector instructions alone take 187, with LDS reads 202, with the products
// 245, with all but global loads 265. 64 columns a workgroup took 392, eight waves 379, three waves a SIMD 425.
//
// Four waves of 32 rows, NT tiles of 32 columns; groups of 32 << SH. (Two workgroups a
// compute unit: with at most 256 registers a wave products' results stay out of the
// accumulator registers, from which each would have to be copied.)
//
// A step is one tile and run: four products and the sums of their results. Steps go tile by
// tile, so only one tile has a group's sum beside its total. A step issues the products of
// the next one between its own sums, so results have the time of 16 sums to come. The next
// chunk's columns come through registers, half of them at a time: loads that go straight
// into LDS would have every later read of LDS wait for them.
//
// Scales and zeros are gathered, a row a lane, which costs the loads' path as much as 1 KB of
// columns each time: kKept groups at once.
constexpr int kKept = 8;

// LONG: rows of several stretches (4096 x 14336, groups of 32, 2047 columns: 452 us, 435 as one
// sum). Those that one sum takes keep a kernel without (a check a chunk costs them 1 to 3%).
template <int NT, int SH, bool Z, bool LONG>
__global__ __launch_bounds__(256, 2) void q4_mfma_kernel(const Q4Args g, const Laid l)
{
    // a chunk's operands and d: [tile][run]; two of each
    constexpr int W = 4;  // waves
    constexpr int kOps = kChunkRuns * kOperand;
    constexpr int kDs = kChunkRuns * kTileCols;
    constexpr int kGroupRuns = 1 << SH;
    constexpr int kGroups = kChunkRuns / kGroupRuns;
    __shared__ __attribute__((aligned(16))) char ops[2][NT * kOps];
    __shared__ float ds[2][NT * kDs];
    // a wave's scales and zeros of kKept groups, those in use and the next ones
    __shared__ __attribute__((aligned(8))) uint16_t kept_scales[W][2][kKept][32];
    __shared__ int8_t kept_zeros[W][2][kKept][32];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int h = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (32 * W) + wave * 32;
    const int tile0 = blockIdx.y * NT;
    const int groups = g.nb >> SH;
    auto row_of = [&](int i) { return n0 + i < g.m.N ? n0 + i : g.m.N - 1; };
    const int chunks = l.runs / kChunkRuns;

    // columns on their way: half of a chunk's pieces of 16 bytes, and d
    constexpr int kPieces = NT * 4 / W;
    constexpr int kDPieces = (NT * 2 + W - 1) / W;
    u32x4 on_way[kPieces];
    float d_on_way[kDPieces];
    const int tiles = l.tiles - tile0 < NT ? l.tiles - tile0 : NT;
    const __amdgpu_buffer_rsrc_t columns = make_rsrc(
        l.ops + (size_t)tile0 * l.runs * kOperand, (uint64_t)tiles * l.runs * kOperand);
    const float *const all_d = l.d + (size_t)tile0 * l.runs * kTileCols;
    auto chunk_of = [&](int t, int chunk) {  // (tiles behind the last are read from the last)
        return (t < tiles ? t : tiles - 1) * chunks + chunk;
    };
    auto load = [&](int chunk, int part) {
#pragma unroll
        for (int i = 0; i < kPieces; i++) {
            const int at = (part * kPieces + i) * W * 1024;  // of the tiles' chunks in a row
            on_way[i] = __builtin_amdgcn_raw_buffer_load_b128(
                columns, threadIdx.x * 16, chunk_of(at / kOps, chunk) * kOps + at % kOps, 0);
        }
        if (part == 0) {
#pragma unroll
            for (int i = 0; i < kDPieces; i++) {
                const int t = i * (W / 2) + (wave >> 1);  // two waves a tile
                if ((i + 1) * (W / 2) <= NT || t < NT)
                    d_on_way[i] = all_d[chunk_of(t, chunk) * kDs + (threadIdx.x & 127u)];
            }
        }
    };
    auto store = [&](int buf, int part) {
#pragma unroll
        for (int i = 0; i < kPieces; i++)
            *reinterpret_cast<u32x4 *>(ops[buf] + (part * kPieces + i) * W * 1024 +
                                       threadIdx.x * 16) = on_way[i];
        if (part == 0) {
#pragma unroll
            for (int i = 0; i < kDPieces; i++)
                if ((i + 1) * (W / 2) <= NT || i * (W / 2) + (wave >> 1) < NT)
                    ds[buf][i * W * 64 + threadIdx.x] = d_on_way[i];
        }
    };

    // A chunk's codes of a lane's two rows, a chunk ahead: lanes of group h hold run h. (Rows
    // behind the last are zeros; runs behind a row's last meet columns of zero.)
    const int64_t rows = g.m.N - n0 < 32 ? g.m.N - n0 : 32;
    const __amdgpu_buffer_rsrc_t codes =
        make_rsrc(static_cast<const char *>(g.m.codes) + n0 * g.nb * 16,
                  rows > 0 ? (uint64_t)rows * g.nb * 16 : 0);
    u32x4 next[2];
    auto fetch = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            next[i] = __builtin_amdgcn_raw_buffer_load_b128(
                codes, ((16 * i + (lane & 15)) * g.nb + h) * 16, chunk * (kChunkRuns * 16), 0);
    };
    // Half a period's scales and zeros of row lane % 32; none behind the row's end.
    uint64_t scales_on_way;
    uint32_t zeros_on_way;
    auto gather = [&](int period) {
        const int at = period * kKept + lane / 32 * (kKept / 2);
        const int64_t place = row_of(lane & 31) * groups + at;
        const uint16_t *sp = static_cast<const uint16_t *>(g.m.scales) + place;
        scales_on_way = 0;
        zeros_on_way = 0;
        if (at + 4 <= groups) {
            __builtin_memcpy(&scales_on_way, sp, 8);
            if constexpr (Z)
                __builtin_memcpy(&zeros_on_way, g.m.zeros + place, 4);
        } else {
            for (int i = 0; at + i < groups; i++) {
                scales_on_way |= (uint64_t)sp[i] << (16 * i);
                if constexpr (Z)
                    zeros_on_way |= (uint32_t)(uint8_t)g.m.zeros[place + i] << (8 * i);
            }
        }
    };
    auto keep = [&](int period) {
#pragma unroll
        for (int i = 0; i < kKept / 2; i++) {
            const int at = lane / 32 * (kKept / 2) + i;
            kept_scales[wave][period & 1][at][lane & 31] = (uint16_t)(scales_on_way >> (16 * i));
            if constexpr (Z)
                kept_zeros[wave][period & 1][at][lane & 31] = (int8_t)(zeros_on_way >> (8 * i));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    int zero[kGroups][2] = {};  // of the next chunk, for a lane's two rows
    auto zeros_of = [&](int chunk) {
        if constexpr (Z) {
#pragma unroll
            for (int i = 0; i < kGroups; i++) {
                const int at = chunk * kGroups + i;
#pragma unroll
                for (int j = 0; j < 2; j++)
                    zero[i][j] = kept_zeros[wave][at / kKept & 1][at % kKept][16 * j + (lane & 15)];
            }
        }
    };

    constexpr int kSteps = kChunkRuns * NT;
    // [tile][row tile, column half], four rows each
    f32x4 acc[NT][4] = {}, part[4], v[2][4];
    float sv[kGroups][2][4];  // scales of the rows that a lane's results are of
    f16x8 a[kChunkRuns][2], b[2][2];  // a chunk's codes; columns of a step and the next
    float d[3][2];
    // the next chunk's codes: lanes of group h hold run h; exchanged, register r holds dword
    // h of run r
    auto exchange = [&](u32x4 &c) {
        auto p = __builtin_amdgcn_permlane32_swap(c.x, c.z, false, false);
        auto q = __builtin_amdgcn_permlane32_swap(c.y, c.w, false, false);
        auto x = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
        auto y = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
        c = u32x4{x[0], x[1], y[0], y[1]};
    };
    auto unpack = [&](int r) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t w = next[i][r];
            const _Float16 z = (_Float16)(float)zero[r / kGroupRuns][i];
            a[r][i] = codes_of(w, f16x2{(_Float16)-1032.0f, (_Float16)-1032.0f} - f16x2{z, z},
                               f16x2{(_Float16)-72.0f, (_Float16)-72.0f} - f16x2{z, z});
        }
    };
    const int begin = (int)((int64_t)chunks * blockIdx.z / gridDim.z);
    const int end = (int)((int64_t)chunks * (blockIdx.z + 1) / gridDim.z);
    float *const y = gridDim.z > 1 ? l.sums + (size_t)blockIdx.z * g.T * g.m.N : g.y;
    // The tile's sums to y, or added to those of the stretches before, by the thread that wrote
    // them.
    auto put = [&](bool first) {
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const int64_t col = (int64_t)(tile0 + t) * kTileCols + 16 * (m & 1) + (lane & 15);
                if (col >= g.T)
                    continue;
                const int64_t n = n0 + 16 * (m >> 1) + 4 * h;
                float *const to = y + col * g.m.N + n;
                if (LONG && n + 4 <= g.m.N) {
                    f32x4 v = acc[t][m];
                    if (!first) {
                        f32x4 before;
                        __builtin_memcpy(&before, to, 16);
                        v = before + v;
                    }
                    __builtin_memcpy(to, &v, 16);
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (n + i < g.m.N)
                        to[i] = !LONG || first ? acc[t][m][i] : to[i] + acc[t][m][i];
            }
    };
    constexpr int kPeriod = kKept / kGroups;  // chunks
    fetch(begin);
    gather(begin / kPeriod);
    load(begin, 0);
    keep(begin / kPeriod);
    gather(begin / kPeriod + 1);
    store(0, 0);
    load(begin, 1);
    store(0, 1);
    zeros_of(begin);
    exchange(next[0]);
    exchange(next[1]);
#pragma unroll
    for (int r = 0; r < kChunkRuns; r++)
        unpack(r);
    for (int chunk = begin; chunk < end; chunk++) {
        const int buf = (chunk - begin) & 1;
        const int after = chunk + 1 < end ? chunk + 1 : chunk;  // (the last one again)
        __syncthreads();
        auto read = [&](int s) {  // a step's columns
            const int t = s / kChunkRuns, r = s % kChunkRuns;
            const char *op = ops[buf] + t * kOps + r * kOperand + lane * 16;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                b[s & 1][i] = *reinterpret_cast<const f16x8 *>(op + 1024 * i);
                d[s % 3][i] = ds[buf][t * kDs + r * kTileCols + 16 * i + (lane & 15)];
            }
        };
        read(0);
        read(1);
        if (chunk % kPeriod == kPeriod - 1) {
            keep(chunk / kPeriod + 1);
            gather(chunk / kPeriod + 2);
        }
#pragma unroll
        for (int i = 0; i < kGroups; i++) {
            const int at = chunk * kGroups + i;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(
                    &kept_scales[wave][at / kKept & 1][at % kKept][16 * j + 4 * h]);
                sv[i][j][0] = f16_bits_to_f32(x[0] & 0xffff), sv[i][j][1] = f16_bits_to_f32(x[0] >> 16);
                sv[i][j][2] = f16_bits_to_f32(x[1] & 0xffff), sv[i][j][3] = f16_bits_to_f32(x[1] >> 16);
            }
        }
        fetch(after);
        load(after, 0);
#pragma unroll
        for (int m = 0; m < 4; m++)
            v[0][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[0][m >> 1], b[0][m & 1], f32x4{}, 0,
                                                            0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kSteps; s++) {
            const int t = s / kChunkRuns, r = s % kChunkRuns, u = s + 1;
            if (s == kSteps / 2) {
                store(buf ^ 1, 0);
                load(after, 1);
            }
            if (t == NT - 1 && r == 0) {
                exchange(next[0]);
                exchange(next[1]);
                zeros_of(after);
            }
#pragma unroll
            for (int m = 0; m < 4; m++) {
                if (u < kSteps)
                    v[u & 1][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        a[u % kChunkRuns][m >> 1], b[u & 1][m & 1], f32x4{}, 0, 0, 0);
                if (m == 0 && s + 2 < kSteps)
                    read(s + 2);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float x = v[s & 1][m][i], e = d[s % 3][m & 1];
                    const float scale = sv[r / kGroupRuns][m >> 1][i];
                    if constexpr (SH == 0) {
                        acc[t][m][i] = fmaf(scale, x * e, acc[t][m][i]);
                    } else {
                        part[m][i] = r % kGroupRuns ? fmaf(x, e, part[m][i]) : x * e;
                        if ((r + 1) % kGroupRuns == 0)
                            acc[t][m][i] = fmaf(scale, part[m][i], acc[t][m][i]);
                    }
                }
                // the next chunk's run in the place of one whose products are all issued
                if (t == NT - 1 && m == 3)
                    unpack(r);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        store(buf ^ 1, 1);
        if constexpr (LONG) {
            if ((chunk + 1 - begin) % l.stretch == 0 && chunk + 1 < end) {
                put(chunk + 1 - begin == l.stretch);
#pragma unroll
                for (int i = 0; i < NT * 4; i++)
                    acc[i / 4][i % 4] = f32x4{};
            }
        }
    }
    put(!LONG || end - begin <= l.stretch);
}

// y = the parts' sums, in their order.
__global__ __launch_bounds__(256) void q4_parts_kernel(const float *__restrict__ sums,
                                                       float *__restrict__ y, int64_t n, int parts)
{
    const int64_t i = block_of_grid() * 256 + threadIdx.x;
    if (i >= n)
        return;
    float v = sums[i];
    for (int p = 1; p < parts; p++)
        v += sums[p * n + i];
    y[i] = v;
}

template <int NT, int SH>
int launch_mfma_group(const Q4Args &g, const Laid &l, hipStream_t stream)
{
    const dim3 grid((unsigned)((g.m.N + 127) / 128), (unsigned)((l.tiles + NT - 1) / NT),
                    (unsigned)l.parts);
    const int chunks = l.runs / kChunkRuns;
    const bool several = l.stretch < (chunks + l.parts - 1) / l.parts;
    auto run = [&](auto *kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, g, l);
        return check_launch();
    };
    if (g.m.zeros)
        return several ? run(q4_mfma_kernel<NT, SH, true, true>)
                       : run(q4_mfma_kernel<NT, SH, true, false>);
    return several ? run(q4_mfma_kernel<NT, SH, false, true>)
                   : run(q4_mfma_kernel<NT, SH, false, false>);
}

template <int NT>
int launch_mfma(const Q4Args &g, const Laid &l, hipStream_t stream)
{
    hipLaunchKernelGGL(q4_columns_kernel, dim3((unsigned)((l.runs + 7) / 8), (unsigned)l.tiles),
                       dim3(256), 0, stream, g.a, l, g.T, g.nb);
    if (int rc = check_launch())
        return rc;
    if (int rc = g.shift == 0   ? launch_mfma_group<NT, 0>(g, l, stream)
                 : g.shift == 1 ? launch_mfma_group<NT, 1>(g, l, stream)
                                : launch_mfma_group<NT, 2>(g, l, stream))
        return rc;
    if (l.parts == 1)
        return BQM_OK;
    const int64_t n = g.T * g.m.N;
    hipLaunchKernelGGL(q4_parts_kernel, grid_of((n + 255) / 256), dim3(256), 0, stream, l.sums,
                       g.y, n, l.parts);
    return check_launch();
}

// ---- a few columns: the matrix cores, all columns in LDS -------------------------------
//
// Up to 32 columns that fit in LDS stay there, as int8 operands, and every wave goes through
// rows by itself, without a barrier between its loads: what counts is bytes on their way, then
// issue (150 instructions for four runs). 100003 x 4096: 9 columns 49 us, 17 60 (the matrix
// alone 42; by tiles 108), 72 with whole tiles dealt to waves; 4096 x 4096 and 9 columns 7.2.
// A code in the high half of its byte is 16 times the code, so an operand takes three
// instructions; a zero's share goes into the products' start, -16 * zero * sum of q. The
// products' rows are columns of the call and their columns rows of the matrix: a lane's
// results are all of one row, whose scales and zeros it loads itself.

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

// LDS of a run's 16 columns: q [64][8 bytes], d [16] fp16, sums of q [16] int16
constexpr int kFewRun = 512 + 32 + 32;

size_t few_lds(int ct, int nb) { return (size_t)((nb + 3) / 4 * 4) * ct * kFewRun; }

// W waves of 16 rows, CT tiles of 16 columns, groups of 32 << SH. A workgroup has an even
// share of the row tiles, and a wave an even share of the runs of those, one after another
// (in periods of four groups): the end of a tile that the wave before it began, whole tiles,
// the beginning of one that others end, whose parts are added at last, in their order.
//
// LONG: one tile of columns leaves room for 284 runs. In groups of 32 that is more roundings of
// one sum than the bound allows (see stretch_of), so a part's first chunks have a sum of their
// own: 1 + 144 + 1 roundings, and 15 at most where waves' parts are added. Shorter rows do without
// (2% of 9 columns' time).
template <int CT, int W, int SH, bool Z, bool LONG>
__global__ __launch_bounds__(64 * W) void q4_few_kernel(const Q4Args g, int tiles)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int kGroupRuns = 1 << SH;
    constexpr int kGroups = 4 / kGroupRuns;  // of a chunk of four runs
    constexpr int kAhead = 3;                // chunks of codes on their way
    constexpr int kPeriod = 4 / kGroups;     // chunks of four groups
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane & 15, h = lane >> 4;
    const int chunks = (g.nb + 3) / 4, groups = g.nb >> SH;
    const int tile0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
    const int own_tiles = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x) - tile0;
    const int periods = (chunks + kPeriod - 1) / kPeriod;  // of a tile
    // (below 2^31: rows are short where they are many)
    auto share = [&](int w) { return (int)((uint32_t)(own_tiles * periods * w) / W); };
    const int share_end = share(wave + 1);
    int at = share(wave), tile = (int)((uint32_t)(own_tiles * wave) / W);

    // The next part of a tile: the period behind the tile's last, chunks.
    int tile_end, first, end;
    __amdgpu_buffer_rsrc_t codes;
    int64_t n0;
    u32x4 next[kAhead];
    auto fetch = [&](int slot, int chunk) {  // lanes of group h: run h
        next[slot] =
            __builtin_amdgcn_raw_buffer_load_b128(codes, (c * g.nb + h) * 16, chunk * 64, 0);
    };
    // Scales and zeros of a tile's rows, which each cost the loads' path as much as 256 bytes
    // of codes: a lane has four groups of row c at once (none behind the row's end), and
    // those of group h the h-th four of sixteen. In use: four groups, the same in all.
    uint64_t scales, scales_held, scales_next;
    uint32_t zeros, zeros_held, zeros_next;
    auto gather = [&](int sixteen) {
        const int64_t n = n0 + c;
        const int at = 16 * sixteen + 4 * h;
        scales_next = 0;
        zeros_next = 0;
        if (n >= g.m.N)
            return;
        const uint16_t *sp = static_cast<const uint16_t *>(g.m.scales) + n * groups + at;
        const int8_t *zp = g.m.zeros + n * groups + at;
        if (at + 4 <= groups) {
            __builtin_memcpy(&scales_next, sp, 8);
            if constexpr (Z)
                __builtin_memcpy(&zeros_next, zp, 4);
        } else {
            for (int k = 0; at + k < groups; k++) {
                scales_next |= (uint64_t)sp[k] << (16 * k);
                if constexpr (Z)
                    zeros_next |= (uint32_t)(uint8_t)zp[k] << (8 * k);
            }
        }
    };
    auto take = [&](int period, bool fresh) {
        if ((period & 3) == 0 || fresh) {
            scales_held = scales_next;
            zeros_held = zeros_next;
            gather((period >> 2) + 1);
        }
        const int from = 4 * (16 * (period & 3) + c);
        const uint32_t lo = __builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)scales_held);
        const uint32_t hi = __builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)(scales_held >> 32));
        scales = (uint64_t)hi << 32 | lo;
        if constexpr (Z)
            zeros = __builtin_amdgcn_ds_bpermute(from, (int)zeros_held);
    };
    auto begin = [&]() {  // the first loads of what is left from `at` on
        tile_end = (tile + 1) * periods;
        const int part_end = (share_end < tile_end ? share_end : tile_end) - tile * periods;
        first = (at - tile * periods) * kPeriod;
        end = part_end * kPeriod < chunks ? part_end * kPeriod : chunks;
        n0 = (int64_t)(tile0 + tile) * 16;
        const int64_t rows = g.m.N - n0 < 16 ? g.m.N - n0 : 16;
        codes = make_rsrc(static_cast<const char *>(g.m.codes) + n0 * g.nb * 16,
                          (uint64_t)rows * g.nb * 16);
#pragma unroll
        for (int i = 0; i < kAhead; i++)
            fetch(i, first + i);
        gather(first / kPeriod / 4);
    };
    if (at < share_end)
        begin();

    // the columns: a thread a column's run
    for (int i = threadIdx.x; i < chunks * 4 * CT * 16; i += 64 * W) {
        const int col = i & 15, run = i >> 4 & 3, t = (i >> 6) % CT, b = i / (64 * CT) * 4 + run;
        uint32_t q[8] = {}, d = 0;
        int sum = 0;
        if (16 * t + col < g.T && b < g.nb) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(
                g.a + ((int64_t)(16 * t + col) * g.nb + b) * kQ81BlockBytes);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                q[k] = p[k];
                sum = sdot4(q[k], 0x01010101u, sum);
            }
            d = p[8];
        }
        char *to = lds + (b * CT + t) * kFewRun;
#pragma unroll
        for (int k = 0; k < 4; k++)
            *reinterpret_cast<u32x2 *>(to + (k * 16 + col) * 8) = u32x2{q[k], q[k + 4]};
        *reinterpret_cast<uint16_t *>(to + 512 + col * 2) = (uint16_t)d;
        *reinterpret_cast<int16_t *>(to + 544 + col * 2) = (int16_t)sum;
    }
    __syncthreads();

    auto store = [&](const float (&v)[CT][4], int64_t row0) {
        const int64_t n = row0 + c;
#pragma unroll
        for (int t = 0; t < CT; t++)
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int col = 16 * t + 4 * h + k;
                if (n < g.m.N && col < g.T)
                    g.y[(int64_t)col * g.m.N + n] = v[t][k];
            }
    };
    float acc[CT][4], sums[CT][4], head[CT][4] = {};  // head: of a tile that another wave began
    bool tail = false;                                // acc: of one that others end
    constexpr int kFirstSum = 36;  // chunks, of 71 at most
    static_assert(kFirstSum % kAhead == 0);
    float before[4];
    while (at < share_end) {
#pragma unroll
        for (int i = 0; i < CT * 4; i++)
            acc[i / 4][i % 4] = 0.0f;
        for (int start = first; start < end; start += kAhead) {
            if constexpr (LONG) {
                if (start - first == kFirstSum) {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        before[k] = acc[0][k];
                        acc[0][k] = 0.0f;
                    }
                }
            }
#pragma unroll
            for (int slot = 0; slot < kAhead; slot++) {
                const int chunk = start + slot;
                if (chunk >= end)
                    break;
                if (chunk % kPeriod == 0)
                    take(chunk / kPeriod, chunk == first);
                // exchanged, register r holds dword h of run r
                auto x = __builtin_amdgcn_permlane32_swap(next[slot][0], next[slot][2], false, false);
                auto y = __builtin_amdgcn_permlane32_swap(next[slot][1], next[slot][3], false, false);
                auto p = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
                auto q = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
                const uint32_t w[4] = {p[0], p[1], q[0], q[1]};
                fetch(slot, chunk + kAhead);  // (behind the part: not used)
#pragma unroll
                for (int j = 0; j < kGroups; j++) {
                    const int at4 = kGroups == 4 ? j : (chunk * kGroups + j) & 3;
                    const float scale =
                        f16_bits_to_f32((uint32_t)(scales >> (16 * at4)) & 0xffffu) * 0.0625f;
                    const int zero = Z ? -16 * (int)(int8_t)(zeros >> (8 * at4)) : 0;
#pragma unroll
                    for (int r = j * kGroupRuns; r < (j + 1) * kGroupRuns; r++) {
                        const uint32_t lo = (w[r] << 4) & 0xf0f0f0f0u, hi = w[r] & 0xf0f0f0f0u;
#pragma unroll
                        for (int t = 0; t < CT; t++) {
                            const char *from = lds + ((chunk * 4 + r) * CT + t) * kFewRun;
                            const long q8 = *reinterpret_cast<const long *>(from + lane * 8);
                            const f16x4 d = *reinterpret_cast<const f16x4 *>(from + 512 + h * 8);
                            i32x4 v = {0, 0, 0, 0};
                            if constexpr (Z) {
                                const i16x4 of_q = *reinterpret_cast<const i16x4 *>(from + 544 + h * 8);
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    v[k] = __mul24(zero, (int)of_q[k]);
                            }
                            v = __builtin_amdgcn_mfma_i32_16x16x32_i8(
                                q8, (long)((uint64_t)hi << 32 | lo), v, 0, 0, 0);
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const float s = (float)v[k], e = (float)d[k];
                                sums[t][k] = r % kGroupRuns ? fmaf(s, e, sums[t][k]) : s * e;
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < CT; t++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            acc[t][k] = fmaf(scale, sums[t][k], acc[t][k]);
                }
            }
        }
        if constexpr (LONG) {
            if (end - first > kFirstSum) {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    acc[0][k] = before[k] + acc[0][k];
            }
        }
        const bool begun = first == 0;
        const int64_t n1 = n0;
        tail = begun && share_end < tile_end;
        at = share_end < tile_end ? share_end : tile_end;
        tile++;
        if (at < share_end)
            begin();
        if (!begun) {
#pragma unroll
            for (int i = 0; i < CT * 4; i++)
                head[i / 4][i % 4] = acc[i / 4][i % 4];
        } else if (!tail) {
            store(acc, n1);
        }
    }
    if (own_tiles % W == 0)
        return;  // (no tile is shared)
    __syncthreads();  // the columns are done with
    float *const heads = reinterpret_cast<float *>(lds) + wave * CT * 4 * 64 + lane;
#pragma unroll
    for (int i = 0; i < CT * 4; i++)
        heads[i * 64] = head[i / 4][i % 4];
    __syncthreads();
    if (!tail)
        return;
    int others = W - 1 - wave;
    if (own_tiles > 1) {  // (counting takes 0.3 us)
        others = 0;
        while (wave + others + 1 < W && share(wave + others + 1) < tile_end)
            others++;
    }
#pragma unroll 4
    for (int o = 1; o <= others; o++)
#pragma unroll
        for (int i = 0; i < CT * 4; i++)
            acc[i / 4][i % 4] += heads[(o * CT * 4 + i) * 64];
    store(acc, n0);
}

// Groups of one sum: the roundings of a group (4 at most) and of 15 parts' additions beside them.
// Two tiles of columns have at most 140 runs, one tile's 284 are at most 142 groups of 64 or 128.
constexpr int kFewOneSum = kMostRoundings - 4 - 15;
static_assert(kLdsMax / (4 * kFewRun) * 4 / 2 <= kFewOneSum);

template <int CT, int W, int SH>
int launch_few_group(const Q4Args &g, hipStream_t stream)
{
    const int tiles = (int)((g.m.N + 15) / 16);
    const int grid = std::min(tiles, compute_units());
    const size_t bytes = std::max(few_lds(CT, g.nb), (size_t)W * 64 * CT * 16);
    auto run = [&](auto *kernel) {
        allow_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes);
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * W), bytes, stream, g, tiles);
        return check_launch();
    };
    if constexpr (CT == 1 && SH == 0) {
        if (g.nb > kFewOneSum)
            return g.m.zeros ? run(q4_few_kernel<CT, W, SH, true, true>)
                             : run(q4_few_kernel<CT, W, SH, false, true>);
    }
    return g.m.zeros ? run(q4_few_kernel<CT, W, SH, true, false>)
                     : run(q4_few_kernel<CT, W, SH, false, false>);
}

template <int CT, int W>
int launch_few_waves(const Q4Args &g, hipStream_t stream)
{
    return g.shift == 0   ? launch_few_group<CT, W, 0>(g, stream)
           : g.shift == 1 ? launch_few_group<CT, W, 1>(g, stream)
                          : launch_few_group<CT, W, 2>(g, stream);
}

// Sixteen waves where a workgroup has at least seven tiles: of 4096 values a row and 17 columns
// 100003 rows take 64 us, with eight waves 75, 32000 rows 26 and 27; 14336 rows 17.6 and 17.9,
// but with 9 columns 12.7 and 12.3, 20000 rows of 512 values 5.8 and 5.4; 4096 rows 12.4 and 9.9.
template <int CT>
int launch_few(const Q4Args &g, hipStream_t stream)
{
    return g.m.N >= (int64_t)compute_units() * 112 ? launch_few_waves<CT, 16>(g, stream)
                                                   : launch_few_waves<CT, 8>(g, stream);
}

bool few_supported(int64_t T, int nb)
{
    return T <= 32 && few_lds(T <= 16 ? 1 : 2, nb) <= kLdsMax;
}

constexpr int kDotCols = 2;       // the most columns without the matrix cores
constexpr int64_t kMostCols = 8192;  // laid out at once

}  // namespace

static int shift_of(int group) { return group == 32 ? 0 : group == 64 ? 1 : 2; }

// What the largest call of up to T columns needs, so that a workspace serves smaller calls too:
// columns laid out grow with T, but parts are the more the fewer columns there are, so those calls
// are looked at whose columns are the most that get their number of parts. (The last turn of
// several may be such a call as well.)
size_t mm_q4_workspace(int64_t N, int64_t T, int64_t K, int group)
{
    const int64_t nb = K / 32;
    if (T <= kDotCols || few_supported(T, (int)nb))
        return 0;
    const int shift = shift_of(group);
    T = std::min(T, kMostCols);
    size_t need = laid_out_bytes(N, T, nb, shift);
    constexpr int64_t kFour = 4 * kTileCols;  // columns that count alike in parts_of
    for (int64_t parts = 16; parts > 2; parts--) {
        const int64_t most = 512 / ((N + 127) / 128 * parts) * kFour;
        if (most > 0)
            need = std::max(need, laid_out_bytes(N, std::min(T, most), nb, shift));
    }
    return need;
}

int launch_mm_q4(const bqm_q4_matrix *m, const void *a, float *y, int64_t T, void *workspace,
                 hipStream_t stream)
{
    Q4Args g = {*m, static_cast<const uint8_t *>(a), y, T, (int)(m->K / 32),
                shift_of(m->group)};
    if (T == 1)
        return launch_dot<1, 4>(g, stream);
    if (T <= kDotCols)
        return launch_dot<2, 4>(g, stream);
    if (few_supported(T, g.nb))
        return T <= 16 ? launch_few<1>(g, stream) : launch_few<2>(g, stream);
    for (int64_t t = 0; t < T; t += kMostCols) {
        g.T = std::min(T - t, kMostCols);
        g.a = static_cast<const uint8_t *>(a) + t * g.nb * kQ81BlockBytes;
        g.y = y + t * m->N;
        const Laid l = laid_out(workspace, m->N, g.T, g.nb, g.shift);
        const int rc = g.T <= 32 ? launch_mfma<1>(g, l, stream)
                       : g.T <= 64 ? launch_mfma<2>(g, l, stream)
                                   : launch_mfma<4>(g, l, stream);
        if (rc)
            return rc;
    }
    return BQM_OK;
}

}  // namespace bqm
