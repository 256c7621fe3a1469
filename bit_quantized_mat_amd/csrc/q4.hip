// q4.hip -- matrices kept in 4 bits (layout in include/bqm.h): made from floats,
// and their rows looked up.
//
// A run of 32 values is 16 bytes, byte i holding values i (low half) and i + 16
// (high half): four dwords whose low halves are values 4j .. 4j + 3 and whose high
// halves 16 + 4j .. 19 + 4j, which is how the products meet a Q8_1 block's q.
#include "common.hpp"
#include "launch.hpp"

namespace bqm {

namespace {

constexpr int kQuadXor2 = 0x4e;  // DPP quad_perm [2, 3, 0, 1]

template <class V>
__device__ __forceinline__ void load8(const V *p, float (&x)[8])
{
    V v[8];
#pragma unroll
    for (int i = 0; i < (int)sizeof(V) / 2; i++) {
        const uint4 r = reinterpret_cast<const uint4 *>(p)[i];
        __builtin_memcpy(reinterpret_cast<char *>(v) + 16 * i, &r, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        x[i] = (float)v[i];
}

__device__ __forceinline__ int near8(float v)  // the nearest code, -8 .. 7
{
    const float r = rintf(v);
    return r > 7.0f ? 7 : r > -8.0f ? (int)r : -8;
}

// Four lanes a run of 32 values, lane h holding 8h .. 8h + 7; a group is 4, 8 or 16
// lanes. One pass: extremes over the group by lane exchanges, then the codes. Bound by the
// fp32 quotients, a division a value as the definition has it: 100003 x 4096 bf16 in 363 us
// (2.9 TB/s), once in a matrix's life.
template <class V>
__global__ __launch_bounds__(256) void q4_quantize_kernel(const V *__restrict__ x, uint8_t *codes,
                                                          uint16_t *scales, int8_t *zeros,
                                                          int64_t eights, int group)
{
    const int64_t at = block_of_grid() * 256 + threadIdx.x;
    // (lanes behind the end work on the last group again and store nothing: whole
    // groups, as the end of the values is the end of one)
    const int per = group / 8;
    const bool live = at < eights;
    const int64_t src = live ? at : eights - per + at % per;
    float v[8];
    load8(x + src * 8, v);
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int i = 1; i < 8; i++) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    for (int m = 1; m < per; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m, 64));
        hi = fmaxf(hi, __shfl_xor(hi, m, 64));
    }
    lo = fminf(lo, 0.0f);
    hi = fmaxf(hi, 0.0f);
    // halved before the difference, which may pass fp32's range
    float s = zeros ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.0f;
    const uint32_t bits = f32_to_f16_bits(fminf(s, 65504.0f));
    s = f16_bits_to_f32(bits);
    int z = 0;
    if (zeros && s != 0.0f)
        z = near8(-8.0f - rintf(lo / s));
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int c = s != 0.0f ? near8(rintf(v[i] / s) + (float)z) : 0;
        mine |= (uint32_t)(c & 15) << (4 * i);
    }
    // lanes 0, 1 of a run hold the low halves, lanes 2, 3 the high ones
    const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)mine, kQuadXor2, 0xf, 0xf, true);
    if (live && (threadIdx.x & 2) == 0) {
        uint2 b = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            b.x |= ((mine >> (4 * i)) & 15) << (8 * i) | ((other >> (4 * i)) & 15) << (8 * i + 4);
            b.y |= ((mine >> (16 + 4 * i)) & 15) << (8 * i) |
                   ((other >> (16 + 4 * i)) & 15) << (8 * i + 4);
        }
        *reinterpret_cast<uint2 *>(codes + (at >> 2) * 16 + (at & 1) * 8) = b;
    }
    if (live && at % per == 0) {
        scales[at / per] = (uint16_t)bits;
        if (zeros)
            zeros[at / per] = (int8_t)z;
    }
}

template <class V>
__device__ __forceinline__ void store8(V *p, const float (&x)[8])
{
    V v[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        v[i] = (V)x[i];
#pragma unroll
    for (int i = 0; i < (int)sizeof(V) / 2; i++) {
        uint4 r;
        __builtin_memcpy(&r, reinterpret_cast<char *>(v) + 16 * i, 16);
        reinterpret_cast<uint4 *>(p)[i] = r;
    }
}

// Eight bytes of codes a thread: values 8h .. 8h + 7 and 16 + 8h .. 23 + 8h of a run.
// 1 << lt threads a row, which loop where a row has more pieces than that. Memory bounds it:
// 8191 rows of 4096 to bf16 17.6 us (4.8 TB/s), all of 100003 to fp16 192 to 206 (5.1 to 5.4),
// to fp32 325 (5.7).
template <class V>
__global__ __launch_bounds__(256) void q4_dequantize_kernel(const bqm_q4_matrix m,
                                                            const int32_t *__restrict__ rows,
                                                            V *__restrict__ out, int64_t n_rows,
                                                            float factor, int lt)
{
    const int64_t i = (block_of_grid() << (8 - lt)) + (threadIdx.x >> lt);
    if (i >= n_rows)
        return;
    int64_t row = i;
    if (rows) {
        row = rows[i];
        row = row < 0 ? 0 : row >= m.N ? m.N - 1 : row;
    }
    const int K = (int)m.K, shift = 31 - __builtin_clz(m.group);
    const uint2 *codes = static_cast<const uint2 *>(m.codes) + row * (K / 16);
    const uint16_t *scales = static_cast<const uint16_t *>(m.scales) + row * (K >> shift);
    const int8_t *zeros = m.zeros ? m.zeros + row * (K >> shift) : nullptr;
    for (int p = threadIdx.x & ((1 << lt) - 1); p < K / 16; p += 1 << lt) {
        const uint2 c = codes[p];
        const int k = (p >> 1) * 32 + (p & 1) * 8;
        const float s = f16_bits_to_f32(scales[k >> shift]);
        const int z = zeros ? zeros[k >> shift] : 0;
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t d = j < 4 ? c.x : c.y;
            const int l = (int)(d << (28 - 8 * (j & 3))) >> 28;
            const int h = (int)(d << (24 - 8 * (j & 3))) >> 28;
            lo[j] = s * (float)(l - z) * factor;
            hi[j] = s * (float)(h - z) * factor;
        }
        store8(out + i * K + k, lo);
        store8(out + i * K + k + 16, hi);
    }
}

template <class V>
int launch_rows(const bqm_q4_matrix *m, const int32_t *rows, void *out, int64_t n_rows,
                float factor, hipStream_t stream)
{
    int lt = 1;
    while (lt < 8 && (16 << lt) < m->K)
        lt++;
    const int64_t grid = (n_rows + (256 >> lt) - 1) >> (8 - lt);
    hipLaunchKernelGGL((q4_dequantize_kernel<V>), grid_of(grid), dim3(256), 0, stream, *m, rows,
                       static_cast<V *>(out), n_rows, factor, lt);
    return check_launch();
}

template <class V>
int launch_quantize(const void *x, const bqm_q4_matrix *m, hipStream_t stream)
{
    const int64_t eights = m->N * (m->K / 8);
    hipLaunchKernelGGL((q4_quantize_kernel<V>), grid_of((eights + 255) / 256), dim3(256), 0, stream,
                       static_cast<const V *>(x),
                       static_cast<uint8_t *>(const_cast<void *>(m->codes)),
                       static_cast<uint16_t *>(const_cast<void *>(m->scales)),
                       const_cast<int8_t *>(m->zeros), eights, m->group);
    return check_launch();
}

}  // namespace

int launch_q4_quantize(const void *x, const bqm_q4_matrix *m, int dtype, hipStream_t stream)
{
    if (dtype == BQM_DTYPE_F32)
        return launch_quantize<float>(x, m, stream);
    if (dtype == BQM_DTYPE_F16)
        return launch_quantize<_Float16>(x, m, stream);
    return launch_quantize<__bf16>(x, m, stream);
}

int launch_q4_dequantize(const bqm_q4_matrix *m, const int32_t *rows, void *out, int64_t n_rows,
                         float factor, int out_dtype, hipStream_t stream)
{
    if (out_dtype == BQM_DTYPE_F32)
        return launch_rows<float>(m, rows, out, n_rows, factor, stream);
    if (out_dtype == BQM_DTYPE_F16)
        return launch_rows<_Float16>(m, rows, out, n_rows, factor, stream);
    return launch_rows<__bf16>(m, rows, out, n_rows, factor, stream);
}

}  // namespace bqm
