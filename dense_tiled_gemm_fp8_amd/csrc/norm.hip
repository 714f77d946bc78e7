/*
 * norm.hip -- rows to E4M3 codes with a scale for each block of 128 values, and
 * the root-mean-square norm with the residual's addition before it.
 *
 *   block_quantize_rows_kernel     one scale for 128 values of a row
 *   block_quantize_square_kernel   one scale for 128 x 128 values
 *   rmsnorm_kernel                 h = x + residual, y = h w / sqrt(mean h^2 + eps),
 *                                  as rows, as codes, or both
 *
 * Of a block with a = max |v|: s = a / 448, i = 448 / a, both rounded to fp32 (1
 * where a < 2^-100), and the codes are the nearest to v * i, ties to even.  |v i|
 * is at most 448 (1 + 2^-22), which rounds to 448.
 */
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_value(uint32_t h) { return __builtin_bit_cast(float, h << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float as_bf16(float v) { return (float)(__bf16)v; }

/* Memory takes vectors at any address of whole elements. */
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

/* `left` (at most 8) elements from base[at] on; the others are zero. */
__device__ __forceinline__ void load8(const void *base, int64_t at, int32_t left, bool f32, float (&v)[8])
{
    if (left >= 8) {
        if (f32) {
            const f32x4_any *x = (const f32x4_any *)((const float *)base + at);
            const f32x4_any a = x[0], b = x[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        } else {
            const u32x4_any a = *(const u32x4_any *)((const uint16_t *)base + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = a[j];
                v[2 * j] = bf16_value(w & 0xFFFFu);
                v[2 * j + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (j < left) v[j] = f32 ? ((const float *)base)[at + j] : bf16_value(((const uint16_t *)base)[at + j]);
    }
}

__device__ __forceinline__ void store8(void *base, int64_t at, int32_t left, bool f32, const float (&v)[8])
{
    if (left >= 8) {
        if (f32) {
            f32x4_any *y = (f32x4_any *)((float *)base + at);
            y[0] = f32x4_any{v[0], v[1], v[2], v[3]};
            y[1] = f32x4_any{v[4], v[5], v[6], v[7]};
        } else {
            *(u32x4_any *)((uint16_t *)base + at) =
                u32x4_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= left) continue;
        if (f32)
            ((float *)base)[at + j] = v[j];
        else
            ((__bf16 *)base)[at + j] = (__bf16)v[j];
    }
}

/* Codes of v * inverse at codes[at ..]; a row's start and `at` are multiples of 8. */
__device__ __forceinline__ void store_codes(uint8_t *codes, int64_t at, int32_t left, float inverse, const float (&v)[8])
{
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inverse, v[1] * inverse, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inverse, v[3] * inverse, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inverse, v[5] * inverse, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inverse, v[7] * inverse, hi, true);
    if (left >= 8) {
        *(uint2 *)(codes + at) = make_uint2((uint32_t)lo, (uint32_t)hi);
        return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < left) codes[at + j] = (uint8_t)((uint32_t)(j < 4 ? lo : hi) >> (8 * (j & 3)));
}

/* Value of the lane that CTRL names (a data-parallel-primitive control). */
template <int CTRL>
__device__ __forceinline__ float lane_move(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

/* Largest over 16 neighbours: swaps within pairs and fours, then mirrored eights
 * and sixteens. */
__device__ __forceinline__ float max16(float a)
{
    a = fmaxf(a, lane_move<0xB1>(a));
    a = fmaxf(a, lane_move<0x4E>(a));
    a = fmaxf(a, lane_move<0x141>(a));
    return fmaxf(a, lane_move<0x140>(a));
}

/* Sum over a wavefront, the same in every lane: sixteens as above, then the four of
 * them in order. */
__device__ __forceinline__ float sum64(float a)
{
    a += lane_move<0xB1>(a);
    a += lane_move<0x4E>(a);
    a += lane_move<0x141>(a);
    a += lane_move<0x140>(a);
    const int v = __builtin_bit_cast(int, a);
    float s = 0.0f;
#pragma unroll
    for (int l = 0; l < 64; l += 16) s += __builtin_bit_cast(float, __builtin_amdgcn_readlane(v, l));
    return s;
}

__device__ __forceinline__ float max8(const float (&v)[8], float a)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[j]));
    return a;
}

struct Scale {
    float scale, inverse;
};

__device__ __forceinline__ Scale block_scale(float a)
{
    if (a < 0x1p-100f) return Scale{1.0f, 1.0f};
    return Scale{a / 448.0f, 448.0f / a};
}

} /* namespace */

/* 16 rows and one K block a workgroup, 8 values a lane: a row's 128 values are 256
 * or 512 consecutive bytes, and the scales of 16 rows one run of 64.  100 x 4001 fp32
 * in 2.6 us: a load, a maximum, a store. */
__global__ __launch_bounds__(256) void block_quantize_rows_kernel(BlockQuantParams p)
{
    const int32_t nk = (p.K + 127) >> 7, rb = blockIdx.x / nk, kb = blockIdx.x - rb * nk;
    const int32_t row = rb * 16 + (threadIdx.x >> 4), k = kb * 128 + (threadIdx.x & 15) * 8;
    const int32_t left = row < p.rows ? p.K - k : 0;
    float v[8];
    load8(p.x, (int64_t)row * p.ldx + k, left, p.f32 != 0, v);
    const Scale s = block_scale(max16(max8(v, 0.0f)));
    if (row >= p.rows) return;
    if ((threadIdx.x & 15) == 0) p.q.scales[(int64_t)kb * p.q.lds + row] = s.scale;
    store_codes(p.q.codes, (int64_t)row * p.q.ld + k, left, s.inverse, v);
}

/* One block of 128 x 128 a workgroup, 64 values a lane, held in registers between
 * the maximum and the codes.  Memory bounds it: 8192 x 8192 bf16, 201 MB, in 41.0 us,
 * 4.9 TB/s. */
__global__ __launch_bounds__(256) void block_quantize_square_kernel(BlockQuantParams p)
{
    __shared__ float red[4];
    const int32_t nk = (p.K + 127) >> 7, rb = blockIdx.x / nk, kb = blockIdx.x - rb * nk;
    const int32_t r0 = rb * 128 + (threadIdx.x >> 4), k = kb * 128 + (threadIdx.x & 15) * 8;
    float v[8][8], a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int32_t row = r0 + i * 16;
        load8(p.x, (int64_t)row * p.ldx + k, row < p.rows ? p.K - k : 0, p.f32 != 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max8(v[i], a);
    a = max16(a);
    a = fmaxf(a, __shfl_xor(a, 16, 64));
    a = fmaxf(a, __shfl_xor(a, 32, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    const Scale s = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    if (threadIdx.x == 0) p.q.scales[(int64_t)rb * p.q.lds + kb] = s.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int32_t row = r0 + i * 16;
        if (row < p.rows) store_codes(p.q.codes, (int64_t)row * p.q.ld + k, p.K - k, s.inverse, v[i]);
    }
}

/* T threads a row, NO octets a thread, in registers from the load to the store: one
 * pass over the data.  Every value of a row is loaded before the row's sum is
 * known, and each octet is stored by the thread that loaded it, so that an output may
 * lie over an input.  Memory bounds it: 4096 x 8192 bf16 with residual into codes, 236
 * MB, in 47.7 us, 4.9 TB/s.  One row of 4096 in 2.6 us, 1000 x 777 fp32 in 3.6: a
 * load, a sum over the row, a store. */
template <int T, int NO>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(NormParams p)
{
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    __shared__ float red[T < 256 ? 1 : T / 64];
    const int32_t row = blockIdx.x * ROWS + (T < 256 ? threadIdx.x / T : 0), t = threadIdx.x % T;
    const int32_t width = row < p.rows ? p.width : 0;
    float h[NO][8], r[NO][8], w[NO][8];
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int32_t k = (i * T + t) * 8;
        load8(p.x, row * p.ldx + k, width - k, p.x_f32 != 0, h[i]);
        if (p.residual) load8(p.residual, row * p.ldr + k, width - k, p.r_f32 != 0, r[i]);
        if (p.weight) load8(p.weight, k, width - k, p.w_f32 != 0, w[i]);
    }
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int32_t k = (i * T + t) * 8;
        if (p.residual) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] += r[i][j];
                /* the norm is of what is held in the residual's type */
                if (!p.r_f32) h[i][j] = as_bf16(h[i][j]);
            }
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part = __builtin_fmaf(h[i][j], h[i][j], part);
        total += part;
    }
    total = sum64(total);
    if constexpr (T >= 256) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = total;
        __syncthreads();
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) total += red[i];
    }
    const float by = 1.0f / sqrtf(total / (float)p.width + p.eps);
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int32_t k = (i * T + t) * 8, left = width - k;
        /* the 16 lanes of a block stay together for the maximum */
        if ((i * T + (t & ~15)) * 8 >= width) continue;
        float y[8];
        if (p.sum) store8(p.sum, row * p.lds + k, left, p.r_f32 != 0, h[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = p.weight ? h[i][j] * by * w[i][j] : h[i][j] * by;
        if (p.y) store8(p.y, row * p.ldy + k, left, p.y_f32 != 0, y);
        if (p.q.codes) {
            const Scale s = block_scale(max16(max8(y, 0.0f)));
            if ((t & 15) == 0) p.q.scales[(int64_t)(k >> 7) * p.q.lds + row] = s.scale;
            store_codes(p.q.codes, row * p.q.ld + k, left, s.inverse, y);
        }
    }
}

hipError_t launch_block_quantize(const BlockQuantParams &p, hipStream_t stream)
{
    const int64_t nk = ((int64_t)p.K + 127) / 128, per = p.block_rows == 1 ? 16 : 128;
    const dim3 grid((uint32_t)(nk * ((p.rows + per - 1) / per)));
    if (p.block_rows == 1)
        hipLaunchKernelGGL(block_quantize_rows_kernel, grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL(block_quantize_square_kernel, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_rmsnorm(const NormParams &p, hipStream_t stream)
{
    const uint32_t rows = (uint32_t)p.rows;
    if (p.width <= 512)
        hipLaunchKernelGGL((rmsnorm_kernel<64, 1>), dim3((rows + 3) / 4), dim3(256), 0, stream, p);
    else if (p.width <= 2048)
        hipLaunchKernelGGL((rmsnorm_kernel<256, 1>), dim3(rows), dim3(256), 0, stream, p);
    else if (p.width <= 4096)
        hipLaunchKernelGGL((rmsnorm_kernel<512, 1>), dim3(rows), dim3(512), 0, stream, p);
    else if (p.width <= 8192)
        hipLaunchKernelGGL((rmsnorm_kernel<1024, 1>), dim3(rows), dim3(1024), 0, stream, p);
    else if (p.width <= 16384)
        hipLaunchKernelGGL((rmsnorm_kernel<1024, 2>), dim3(rows), dim3(1024), 0, stream, p);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<1024, 4>), dim3(rows), dim3(1024), 0, stream, p);
    return hipGetLastError();
}

} /* namespace g355 */
