// mm_q4.hip -- product of a 4-bit matrix (layout in include/bqm.h) and Q8_1
// activation columns:
//   y[t][n] = sum_j scale * d_a[t][j] * sum_{i < 32} (code - zero) * q[t][32j + i].
//
// The inner sums are exact whole numbers. A code's nibble kept in the high half of
// its byte is 16 times the code as int8, so the low halves need a shift and a mask
// and the high ones a mask; the 16 goes into d_a.
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

// Columns t0 .. t0 + TC - 1 of runs b0 .. b0 + n - 1, as two planes of 16 bytes a run
// (a lane reads each with one load, neighbours next to each other), d / 16 and sums.
template <int TC>
struct Stage {
    uint4 lo[TC][kStageRuns], hi[TC][kStageRuns];
    float d[TC][kStageRuns];
    int sum[TC][kStageRuns];
};

template <int TC, bool Z>
__device__ __forceinline__ void stage_columns(Stage<TC> &s, const Q4Args &g, int64_t t0, int b0,
                                              int n)
{
    for (int i = threadIdx.x; i < TC * kStageRuns; i += 256) {
        const int t = i / kStageRuns, b = i % kStageRuns;
        if (b >= n)
            continue;
        const int64_t col = t0 + t < g.T ? t0 + t : g.T - 1;
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
// the row's runs in turn.
template <int TC, int R, bool Z>
__global__ __launch_bounds__(256) void q4_dot_kernel(const Q4Args g, int lr)
{
    __shared__ Stage<TC> s;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int per = 64 >> lr;  // rows side by side
    const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * (per * R) + (lane >> lr);
    const int64_t t0 = (int64_t)blockIdx.y * TC;
    float acc[R][TC] = {};
    for (int b0 = 0; b0 < g.nb; b0 += kStageRuns) {
        const int n = g.nb - b0 < kStageRuns ? g.nb - b0 : kStageRuns;
        if (b0)
            __syncthreads();
        stage_columns<TC, Z>(s, g, t0, b0, n);
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
            const float v = row_sum(acc[r][t], lr);
            if ((lane & ((1 << lr) - 1)) == 0 && row < g.m.N && t0 + t < g.T)
                g.y[(t0 + t) * g.m.N + row] = v;
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
    const dim3 grid((unsigned)((g.m.N + rows - 1) / rows), (unsigned)((g.T + TC - 1) / TC));
    if (g.m.zeros)
        hipLaunchKernelGGL((q4_dot_kernel<TC, R, true>), grid, dim3(256), 0, stream, g, lr);
    else
        hipLaunchKernelGGL((q4_dot_kernel<TC, R, false>), grid, dim3(256), 0, stream, g, lr);
    return check_launch();
}

// ---- many columns: the matrix cores ------------------------------------------------
//
// Codes less zeros (-15 .. 15) and q (-127 .. 127) are exact in fp16, and sums over a run
// of 32 are exact in fp32, so a 32 x 32 tile of a run is two 32x32x16 products whose result
// needs one fma by d_a, and one by the scale at the end of a group. Eight codes become
// fp16 in ten instructions: a nibble under the exponent of 1024 is 1024 + nibble.
//
// The columns are laid out once a call, in the order in which lanes read them: an
// operand's 64 lanes x 16 bytes in a row. A lane of half h (lane / 32) takes dwords h and
// h + 2 of a row's run, so its values of product p are 4j + {0, 2}, 16 + 4j + {0, 2},
// 4j + {1, 3}, 16 + 4j + {1, 3} with j = 2p + h.

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileCols = 32;    // columns of a tile
constexpr int kChunkRuns = 4;    // runs between two barriers
constexpr int kOperand = 2048;   // bytes of one tile's run: two operands

// Workspace: operands [column tile][run][2][64][16 bytes], then d [column tile][run][32]
// fp32; runs padded to whole chunks, columns to whole tiles, with zeros.
struct Laid {
    char *ops;
    float *d;
    int runs, tiles;
};

Laid laid_out(void *workspace, int64_t T, int nb)
{
    Laid l;
    l.runs = (nb + kChunkRuns - 1) / kChunkRuns * kChunkRuns;
    l.tiles = (int)((T + kTileCols - 1) / kTileCols);
    l.ops = static_cast<char *>(workspace);
    l.d = reinterpret_cast<float *>(l.ops + (size_t)l.tiles * l.runs * kOperand);
    return l;
}

size_t laid_out_bytes(int64_t T, int64_t nb)
{
    const size_t runs = (nb + kChunkRuns - 1) / kChunkRuns * kChunkRuns;
    return (size_t)((T + kTileCols - 1) / kTileCols) * runs * (kOperand + kTileCols * 4);
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
    char *to = l.ops + ((size_t)tile * l.runs + run) * kOperand + c * 16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint4 v;
        halves_of(q[j], v.x, v.z);
        halves_of(q[j + 4], v.y, v.w);
        *reinterpret_cast<uint4 *>(to + (j >> 1) * 1024 + (j & 1) * 512) = v;
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

// 16 or 4 bytes a lane, straight into LDS at base + that many bytes times lane.
__device__ __forceinline__ void to_lds16(const void *from, void *base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)base, 16, 0, 0);
}

__device__ __forceinline__ void to_lds4(const void *from, void *base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)base, 4, 0, 0);
}

// Four waves of 32 rows, NT tiles of 32 columns; groups of 32 << SH. (Two workgroups a
// compute unit: with at most 256 registers a wave products' results stay out of the
// accumulator registers, from which each would have to be copied.)
template <int NT, int SH, bool Z>
__global__ __launch_bounds__(256, 2) void q4_mfma_kernel(const Q4Args g, const Laid l)
{
    // a chunk's operands and d: [tile][run]; two of each
    constexpr int kOps = kChunkRuns * kOperand;
    constexpr int kDs = kChunkRuns * kTileCols;
    __shared__ __attribute__((aligned(16))) char ops[2][NT * kOps];
    __shared__ float ds[2][NT * kDs];
    __shared__ __attribute__((aligned(16))) float ss[4][kChunkRuns][32];  // a wave's scales
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    const int64_t n0 = (int64_t)blockIdx.x * 128 + wave * 32;
    const int tile0 = blockIdx.y * NT;
    const int64_t row = n0 + (lane & 31) < g.m.N ? n0 + (lane & 31) : g.m.N - 1;
    const uint4 *codes = static_cast<const uint4 *>(g.m.codes) + row * g.nb;
    constexpr int kGroupRuns = 1 << SH;
    const int groups = g.nb >> SH;
    const uint16_t *scales = static_cast<const uint16_t *>(g.m.scales) + row * groups;
    const int8_t *zeros = g.m.zeros + row * groups;
    const int chunks = l.runs / kChunkRuns;

    auto stage = [&](int chunk, int buf) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            // (tiles behind the last are read from the last)
            const int tile = tile0 + t < l.tiles ? tile0 + t : l.tiles - 1;
            const size_t piece = (size_t)tile * chunks + chunk;
            const char *from = l.ops + piece * kOps + wave * 1024;  // 1 KB a wave of each 4
            char *to = ops[buf] + t * kOps + wave * 1024;
            to_lds16(from + lane * 16u, to);
            to_lds16(from + 4096 + lane * 16u, to + 4096);
            if (wave == t)
                to_lds4(l.d + piece * kDs + (uint32_t)lane, ds[buf] + t * kDs);
            if (wave == (t ^ 1))
                to_lds4(l.d + piece * kDs + 64 + (uint32_t)lane, ds[buf] + t * kDs + 64);
        }
    };
    // A chunk's codes, scales and zeros of a lane's row, a chunk ahead: lanes of half h
    // hold runs 2i + h of the chunk's pairs.
    constexpr int kGroups = kChunkRuns / kGroupRuns;
    uint4 next[2];
    uint32_t next_scale[kGroups];
    int next_zero[kGroups];
    auto fetch = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int b = chunk * kChunkRuns + 2 * i + half;
            next[i] = codes[b < g.nb ? b : g.nb - 1];
        }
#pragma unroll
        for (int i = 0; i < kGroups; i++) {
            const int at = chunk * kGroups + i;
            next_scale[i] = at < groups ? scales[at] : 0;  // (runs behind the end count nothing)
            next_zero[i] = Z && at < groups ? zeros[at] : 0;
        }
    };

    // Steps of one run and column tile, run by run: a step issues the products of the
    // next one between its own sums, so results have the time of 16 sums to come, and
    // reads the operands of the one after.
    constexpr int kSteps = kChunkRuns * NT;
    f32x16 acc[NT] = {}, part[NT] = {}, v[2];
    float sv[16] = {};  // scales of the group that `part` is of, for the rows of a lane's results
    uint32_t w[2][4];
    f16x2 low[kGroups], high[kGroups];
    f16x8 a[2][2], b[2];  // codes of a run and the next; columns of the next step
    float d[3];
    auto unpack = [&](int r, int p) {
        // after the swap the lower half holds dword 0 (2) of the pair's first run and
        // the upper half dword 1 (3); the other register the same of the second run
        uint32_t *x = w[r / 2];
        if ((r & 1) == 0) {
            auto y = __builtin_amdgcn_permlane32_swap(x[2 * p], x[2 * p + 1], false, false);
            x[2 * p] = y[0], x[2 * p + 1] = y[1];
        }
        a[r & 1][p] = codes_of(x[2 * p + (r & 1)], low[r / kGroupRuns], high[r / kGroupRuns]);
    };
    auto scales_of = [&](int group) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float4 x =
                *reinterpret_cast<const float4 *>(&ss[wave][group][8 * q + 4 * half]);
            sv[4 * q] = x.x, sv[4 * q + 1] = x.y, sv[4 * q + 2] = x.z, sv[4 * q + 3] = x.w;
        }
    };
    stage(0, 0);
    fetch(0);
    for (int chunk = 0; chunk < chunks; chunk++) {
        const int buf = chunk & 1;
        __syncthreads();
        auto read = [&](int s) {  // a step's columns
            const int r = s / NT, t = s % NT;
            const char *op = ops[buf] + t * kOps + r * kOperand + lane * 16;
            b[0] = *reinterpret_cast<const f16x8 *>(op);
            b[1] = *reinterpret_cast<const f16x8 *>(op + 1024);
            d[s % 3] = ds[buf][t * kDs + r * kTileCols + (lane & 31)];
        };
        read(0);
#pragma unroll
        for (int i = 0; i < 2; i++)
            w[i][0] = next[i].x, w[i][1] = next[i].y, w[i][2] = next[i].z, w[i][3] = next[i].w;
#pragma unroll
        for (int i = 0; i < kGroups; i++) {
            // scales go through LDS to the rows that a lane's results are of
            if (half == 0)
                ss[wave][i][lane] = f16_bits_to_f32(next_scale[i]);
            const _Float16 z = (_Float16)(float)next_zero[i];
            low[i] = f16x2{(_Float16)-1032.0f, (_Float16)-1032.0f} - f16x2{z, z};
            high[i] = f16x2{(_Float16)-72.0f, (_Float16)-72.0f} - f16x2{z, z};
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (chunk + 1 < chunks) {
            stage(chunk + 1, buf ^ 1);
            fetch(chunk + 1);
        }
        if constexpr (SH == 0)
            scales_of(0);
        unpack(0, 0);
        unpack(0, 1);
        v[0] = f32x16{};
        v[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[0][0], b[0], v[0], 0, 0, 0);
        v[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[0][1], b[1], v[0], 0, 0, 0);
        read(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kSteps; s++) {
            const int r = s / NT, t = s % NT, u = s + 1, ur = u / NT;
            auto sums = [&](int from) {
#pragma unroll
                for (int i = from; i < from + 8; i++) {
                    const float x = v[s & 1][i];
                    if constexpr (SH == 0) {
                        acc[t][i] = fmaf(sv[i], x * d[s % 3], acc[t][i]);
                    } else if (r % kGroupRuns) {
                        part[t][i] = fmaf(x, d[s % 3], part[t][i]);
                    } else {  // a group begins: the one before is done
                        acc[t][i] = fmaf(sv[i], part[t][i], acc[t][i]);
                        part[t][i] = x * d[s % 3];
                    }
                }
            };
            // the next run's codes, half of them at a time, before its first step's products
            if (NT == 1 && r + 1 < kChunkRuns) {
                unpack(r + 1, 0);
                unpack(r + 1, 1);
            }
            if (u < kSteps) {
                v[u & 1] = f32x16{};
                v[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[ur & 1][0], b[0], v[u & 1], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            sums(0);
            if (NT > 1 && t == NT - 2 && r + 1 < kChunkRuns)
                unpack(r + 1, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (u < kSteps)
                v[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[ur & 1][1], b[1], v[u & 1], 0, 0, 0);
            if (s + 2 < kSteps)
                read(s + 2);
            __builtin_amdgcn_sched_barrier(0);
            sums(8);
            if (NT > 1 && t == NT - 2 && r + 1 < kChunkRuns)
                unpack(r + 1, 1);
            if (SH == 0 && t == NT - 1 && r + 1 < kChunkRuns)
                scales_of(r + 1);
            if (SH > 0 && t == NT - 1 && (r + 1) % kGroupRuns == 0)
                scales_of(r / kGroupRuns);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (SH > 0) {
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                acc[t][i] = fmaf(sv[i], part[t][i], acc[t][i]);
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t col = (int64_t)(tile0 + t) * kTileCols + (lane & 31);
        if (col >= g.T)
            continue;
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int64_t n = n0 + 8 * q + 4 * half + i;
                if (n < g.m.N)
                    g.y[col * g.m.N + n] = acc[t][4 * q + i];
            }
    }
}

template <int NT, int SH>
int launch_mfma_group(const Q4Args &g, const Laid &l, hipStream_t stream)
{
    const dim3 grid((unsigned)((g.m.N + 127) / 128), (unsigned)((l.tiles + NT - 1) / NT));
    if (g.m.zeros)
        hipLaunchKernelGGL((q4_mfma_kernel<NT, SH, true>), grid, dim3(256), 0, stream, g, l);
    else
        hipLaunchKernelGGL((q4_mfma_kernel<NT, SH, false>), grid, dim3(256), 0, stream, g, l);
    return check_launch();
}

template <int NT>
int launch_mfma(const Q4Args &g, const Laid &l, hipStream_t stream)
{
    hipLaunchKernelGGL(q4_columns_kernel, dim3((unsigned)((l.runs + 7) / 8), (unsigned)l.tiles),
                       dim3(256), 0, stream, g.a, l, g.T, g.nb);
    if (int rc = check_launch())
        return rc;
    return g.shift == 0   ? launch_mfma_group<NT, 0>(g, l, stream)
           : g.shift == 1 ? launch_mfma_group<NT, 1>(g, l, stream)
                          : launch_mfma_group<NT, 2>(g, l, stream);
}

constexpr int kDotCols = 8;       // the most columns without the matrix cores
constexpr int64_t kMostCols = 8192;  // laid out at once

}  // namespace

size_t mm_q4_workspace(int64_t T, int64_t K)
{
    return T <= kDotCols ? 0 : laid_out_bytes(std::min(T, kMostCols), K / 32);
}

int launch_mm_q4(const bqm_q4_matrix *m, const void *a, float *y, int64_t T, void *workspace,
                 hipStream_t stream)
{
    Q4Args g = {*m, static_cast<const uint8_t *>(a), y, T, (int)(m->K / 32),
                m->group == 32 ? 0 : m->group == 64 ? 1 : 2};
    if (T == 1)
        return launch_dot<1, 4>(g, stream);
    if (T == 2)
        return launch_dot<2, 4>(g, stream);
    if (T <= 4)
        return launch_dot<4, 4>(g, stream);
    if (T <= kDotCols)
        return launch_dot<8, 4>(g, stream);
    for (int64_t t = 0; t < T; t += kMostCols) {
        g.T = std::min(T - t, kMostCols);
        g.a = static_cast<const uint8_t *>(a) + t * g.nb * kQ81BlockBytes;
        g.y = y + t * m->N;
        const Laid l = laid_out(workspace, g.T, g.nb);
        const int rc = g.T <= 32 ? launch_mfma<1>(g, l, stream)
                       : g.T <= 64 ? launch_mfma<2>(g, l, stream)
                                   : launch_mfma<4>(g, l, stream);
        if (rc)
            return rc;
    }
    return BQM_OK;
}

}  // namespace bqm
