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

}  // namespace

int launch_mm_q4(const bqm_q4_matrix *m, const void *a, float *y, int64_t T, hipStream_t stream)
{
    const Q4Args g = {*m, static_cast<const uint8_t *>(a), y, T, (int)(m->K / 32),
                      m->group == 32 ? 0 : m->group == 64 ? 1 : 2};
    if (T == 1)
        return launch_dot<1, 4>(g, stream);
    if (T == 2)
        return launch_dot<2, 4>(g, stream);
    return launch_dot<4, 4>(g, stream);
}

}  // namespace bqm
