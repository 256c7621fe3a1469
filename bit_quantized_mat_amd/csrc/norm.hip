// norm.hip -- root-mean-square norm of a token's values, with the residual's
// addition before it and, if asked for, Q8_1 blocks of the result.
//
//   s = x + add (fp32, rounded to the stream's type and kept),
//   r = 1 / sqrt(mean of s^2 + eps), y = fp32(fp32(s * r) * gain).
//
// The mean is formed in fp64: a square of two fp32 values is exact there, so the
// sum's order moves r by less than its rounding to fp32 does, and the 8-bit steps
// that follow fall on the same side of their borders however a row is split.
//
// A row's values stay in registers between the two passes over them, eight
// neighbours a thread (16 bytes of a 16-bit stream), so memory is read once and
// written once; four lanes share a Q8_1 block. Memory bounds it: 9000 rows of 4096 bf16
// with an addend take 55 us (5.4 TB/s; a large copy reaches 5.1), 61 with Q8_1 blocks and a
// fp32 addend (5.5). One row takes 3.0 us: a load, the waves' exchange, a store.
#include "common.hpp"
#include "launch.hpp"
#include "q8_1.hpp"

namespace bqm {

namespace {

struct None {};

struct NormArgs {
    const void *x, *add;
    const float *gain;
    void *sum, *y;
    uint8_t *a;
    int64_t T;
    int K;
    int lanes;  // log2 of a row's lanes: up to 6 within a wave, else
    int waves;  // a row's waves
    double eps;
    int y_dtype;
};

template <class V>
__device__ __forceinline__ void load8(const V *p, float (&x)[8])
{
    V v[8];
    if constexpr (sizeof(V) == 2) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        __builtin_memcpy(v, &r, 16);
    } else {
        const uint4 r = reinterpret_cast<const uint4 *>(p)[0];
        const uint4 s = reinterpret_cast<const uint4 *>(p)[1];
        __builtin_memcpy(v, &r, 16);
        __builtin_memcpy(v + 4, &s, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        x[i] = (float)v[i];
}

template <class V>
__device__ __forceinline__ void store8(V *p, const float (&x)[8])
{
    V v[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        v[i] = (V)x[i];
    uint4 r;
    __builtin_memcpy(&r, v, 16);
    reinterpret_cast<uint4 *>(p)[0] = r;
    if constexpr (sizeof(V) == 4) {
        __builtin_memcpy(&r, v + 4, 16);
        reinterpret_cast<uint4 *>(p)[1] = r;
    }
}

// C: pieces of 512 values a wave holds. A workgroup has blockDim / 64 / waves rows, or, of
// rows of up to 256 values, several a wave (100000 rows of 64 values: 10 us, 36 with a wave each).
template <class S, class A, int C>
__global__ __launch_bounds__(1024) void rms_norm_kernel(const NormArgs g)
{
    __shared__ double part[16];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & ((1 << g.lanes) - 1);
    const int rows = (int)(blockDim.x >> g.lanes) / g.waves;
    const int w = wave % g.waves;
    const int64_t row = block_of_grid() * rows + (threadIdx.x >> g.lanes) / g.waves;
    const bool live = row < g.T;
    const int64_t at = row * g.K;
    float s[C][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int k = ((c * g.waves + w) * 64 + lane) * 8;
        const bool in = live && k < g.K;
#pragma unroll
        for (int i = 0; i < 8; i++)
            s[c][i] = 0.0f;
        if (in)
            load8(static_cast<const S *>(g.x) + at + k, s[c]);
        if constexpr (!__is_same(A, None)) {
            if (in) {
                float b[8];
                load8(static_cast<const A *>(g.add) + at + k, b);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    s[c][i] = (float)(S)(s[c][i] + b[i]);
                store8(static_cast<S *>(g.sum) + at + k, s[c]);
            }
        } else if (g.sum && in) {
            store8(static_cast<S *>(g.sum) + at + k, s[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const double v = (double)s[c][i];
            sum = __builtin_fma(v, v, sum);
        }
    }
    for (int m = 1 << g.lanes >> 1; m; m >>= 1)
        sum += __shfl_xor(sum, m, 64);
    if (g.waves > 1) {
        if (lane == 0)
            part[wave] = sum;
        __syncthreads();
        const int first = wave - w;
        sum = 0.0;
        for (int i = 0; i < g.waves; i++)
            sum += part[first + i];
    }
    const float r = (float)(1.0 / sqrt(sum / (double)g.K + g.eps));
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int k = ((c * g.waves + w) * 64 + lane) * 8;
        const bool in = live && k < g.K;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            y[i] = s[c][i] * r;
        if (g.gain && in) {
            float f[8];
            load8(g.gain + k, f);
#pragma unroll
            for (int i = 0; i < 8; i++)
                y[i] = y[i] * f[i];
        }
        if (g.y && in) {
            if (g.y_dtype == BQM_DTYPE_F32)
                store8(static_cast<float *>(g.y) + at + k, y);
            else if (g.y_dtype == BQM_DTYPE_F16)
                store8(static_cast<_Float16 *>(g.y) + at + k, y);
            else
                store8(static_cast<__bf16 *>(g.y) + at + k, y);
        }
        if (g.a) {  // (every lane: a block's four exchange their parts)
            const Q81Quarter q = q8_1_block_by_4(y);
            if (in) {
                uint32_t *out = reinterpret_cast<uint32_t *>(
                    g.a + (row * (g.K / kQ81BlockElems) + k / kQ81BlockElems) * kQ81BlockBytes);
                const int h = lane & 3;
                out[2 * h] = q.q4[0];
                out[2 * h + 1] = q.q4[1];
                if (h == 0)
                    out[8] = q.field;
            }
        }
    }
}

template <class S, class A>
int launch(const NormArgs &g0, hipStream_t stream)
{
    NormArgs g = g0;
    const int pieces = (g.K + 511) / 512;
    const int c = pieces <= 16 ? 1 : pieces <= 32 ? 2 : pieces <= 64 ? 4 : 8;
    g.waves = (pieces + c - 1) / c;
    g.lanes = 6;
    while (g.K <= 4 << g.lanes)  // (half the lanes hold it)
        g.lanes--;
    const int rows = g.waves >= 4 ? 1 : (256 >> g.lanes) / g.waves;
    const dim3 grid = grid_of((g.T + rows - 1) / rows);
    const dim3 block((unsigned)(rows * g.waves << g.lanes));
    if (c == 1)
        hipLaunchKernelGGL((rms_norm_kernel<S, A, 1>), grid, block, 0, stream, g);
    else if (c == 2)
        hipLaunchKernelGGL((rms_norm_kernel<S, A, 2>), grid, block, 0, stream, g);
    else if (c == 4)
        hipLaunchKernelGGL((rms_norm_kernel<S, A, 4>), grid, block, 0, stream, g);
    else
        hipLaunchKernelGGL((rms_norm_kernel<S, A, 8>), grid, block, 0, stream, g);
    return check_launch();
}

template <class S>
int launch_add(const NormArgs &g, int add_dtype, hipStream_t stream)
{
    if (!g.add)
        return launch<S, None>(g, stream);
    if (add_dtype == BQM_DTYPE_F32)
        return launch<S, float>(g, stream);
    if (add_dtype == BQM_DTYPE_F16)
        return launch<S, _Float16>(g, stream);
    return launch<S, __bf16>(g, stream);
}

}  // namespace

int launch_rms_norm(const void *x, const void *add, const float *gain, void *sum, void *y, void *a,
                    int64_t T, int K, double eps, int dtype, int add_dtype, int y_dtype,
                    hipStream_t stream)
{
    const NormArgs g = {x, add, gain, sum, y, static_cast<uint8_t *>(a), T, K, 6, 1, eps, y_dtype};
    if (dtype == BQM_DTYPE_F32)
        return launch_add<float>(g, add_dtype, stream);
    if (dtype == BQM_DTYPE_F16)
        return launch_add<_Float16>(g, add_dtype, stream);
    return launch_add<__bf16>(g, add_dtype, stream);
}

}  // namespace bqm
