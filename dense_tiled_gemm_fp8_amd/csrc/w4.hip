/*
 * w4.hip -- matrices held in 4 bits with a scale for each group of K, and
 * products of a few bf16 rows with them.
 *
 *   INT    w[n][k] = (u[n][k] - z[n][g]) * s[n][g], u in 0..15, g = k / group,
 *          s bf16, z a byte (8 where there are no zero points)
 *   MXFP4  w[n][k] = e2m1(c[n][k]) * 2^(e[n][k / 32] - 127)
 *
 *   w4_quantize_kernel    8 consecutive elements a thread, the group's range
 *                         by shuffles among its group / 8 threads
 *   w4_dequantize_kernel  8 consecutive elements a thread
 *   w4_gemm_kernel        y[m][n] = sum_k x[m][k] w[n][k]
 */
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_value(uint32_t h) { return __builtin_bit_cast(float, h << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, v);
}

/* 8 elements of a row from k on; those past K read as zero. */
__device__ __forceinline__ void load8_row(const W4QuantParams &p, int32_t n, int32_t k, float (&v)[8])
{
    const int64_t at = (int64_t)n * p.ld + k;
    if (p.vec && k + 8 <= p.w.K) {
        if (p.f32) {
            const float4 a = *(const float4 *)((const float *)p.x + at);
            const float4 b = *(const float4 *)((const float *)p.x + at + 4);
            v[0] = a.x;
            v[1] = a.y;
            v[2] = a.z;
            v[3] = a.w;
            v[4] = b.x;
            v[5] = b.y;
            v[6] = b.z;
            v[7] = b.w;
        } else {
            const uint4 a = *(const uint4 *)((const uint16_t *)p.x + at);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
                v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (k + j < p.w.K)
            v[j] = p.f32 ? ((const float *)p.x)[at + j] : bf16_value(((const uint16_t *)p.x)[at + j]);
    }
}

/* Code of the E2M1 value nearest to v, ties to the even code, magnitudes past
 * 6 to 6.  The borders between neighbouring codes, with a tie's even side:
 * 0.25 down, 0.75 up, 1.25 down, 1.75 up, 2.5 down, 3.5 up, 5 down. */
__device__ __forceinline__ uint32_t encode_e2m1(float v)
{
    const float a = fabsf(v);
    const uint32_t mag = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return mag | ((__builtin_bit_cast(uint32_t, v) >> 28) & 8u);
}

} /* namespace */

/* One thread for 8 elements; the group / 8 threads of a group are neighbours
 * in a wavefront. */
__global__ __launch_bounds__(256) void w4_quantize_kernel(W4QuantParams p)
{
    const int32_t lanes = p.w.group >> 3;                 /* 4, 8 or 16        */
    const int32_t per_row = p.w.ng * lanes;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool in = id < (int64_t)p.w.N * per_row;
    const int32_t n = in ? (int32_t)(id / per_row) : 0;
    const int32_t oct = in ? (int32_t)(id % per_row) : 0;
    const int32_t k = oct * 8;
    float v[8];
    load8_row(p, n, k, v);
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, v[j]);
        hi = fmaxf(hi, v[j]);
    }
    for (int o = lanes >> 1; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, o, 64));
        hi = fmaxf(hi, __shfl_xor(hi, o, 64));
    }
    if (!in || k >= p.w.K) return;
    const int32_t g = oct / lanes;
    const int64_t at = (int64_t)n * p.w.ng + g;
    const bool first = oct % lanes == 0;
    uint32_t word = 0;
    if (p.w.mx) {
        const float a = fmaxf(-lo, hi);
        const uint32_t bits = __builtin_bit_cast(uint32_t, a);
        /* exponent of a less 2, not under 2^-127 (a's own exponent field
         * counts from 127; a subnormal a is under 2^-126) */
        int32_t e = (int32_t)(bits >> 23) - 2;
        e = e < 0 ? 0 : e;
        if (first) ((uint8_t *)p.w.scales)[at] = (uint8_t)e;
#pragma unroll
        for (int j = 0; j < 8; ++j) word |= encode_e2m1(__builtin_ldexpf(v[j], 127 - e)) << (4 * j);
    } else {
        const float range = p.w.zeros ? hi - lo : fmaxf(-lo, hi);
        float s = 1.0f;
        /* the scale itself is held in 16 bits, so codes go by the rounded one */
        if (range >= 0x1p-100f) s = (float)(__bf16)(range / (p.w.zeros ? 15.0f : 7.0f));
        float z = 8.0f;
        if (p.w.zeros) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
        if (first) {
            ((__bf16 *)p.w.scales)[at] = (__bf16)s;
            if (p.w.zeros) p.w.zeros[at] = (uint8_t)z;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = fminf(fmaxf(rintf(v[j] / s) + z, 0.0f), 15.0f);
            word |= (k + j < p.w.K ? (uint32_t)u : 0u) << (4 * j);
        }
    }
    *(uint32_t *)(p.w.codes + (int64_t)n * p.w.ldb + (k >> 1)) = word;
}

__global__ __launch_bounds__(256) void w4_dequantize_kernel(W4QuantParams p)
{
    const int32_t per_row = (p.w.K + 7) >> 3;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (int64_t)p.w.N * per_row) return;
    const int32_t n = (int32_t)(id / per_row);
    const int32_t k = (int32_t)(id % per_row) * 8;
    const uint32_t word = *(const uint32_t *)(p.w.codes + (int64_t)n * p.w.ldb + (k >> 1));
    const int64_t at = (int64_t)n * p.w.ng + k / p.w.group;
    float v[8];
    if (p.w.mx) {
        const uint32_t e = ((const uint8_t *)p.w.scales)[at];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = (word >> (4 * j)) & 15u, m = c & 7u;
            /* magnitude codes 0 and 1 are 0 and 0.5, the others (2 + m % 2)
             * times 2^(m / 2 - 2) */
            const float mag = m < 2 ? 0.5f * (float)m : __builtin_ldexpf((float)(2 + (m & 1u)), (int)(m >> 1) - 2);
            v[j] = e == 255 ? __builtin_nanf("") : __builtin_ldexpf(c & 8u ? -mag : mag, (int)e - 127);
        }
    } else {
        const float s = bf16_value(((const uint16_t *)p.w.scales)[at]);
        const float z = p.w.zeros ? (float)p.w.zeros[at] : 8.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((float)((word >> (4 * j)) & 15u) - z) * s;
    }
    const int64_t o = (int64_t)n * p.ld + k;
    if (p.vec && k + 8 <= p.w.K) {
        if (p.f32) {
            *(float4 *)((float *)p.y + o) = make_float4(v[0], v[1], v[2], v[3]);
            *(float4 *)((float *)p.y + o + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *(uint4 *)((uint16_t *)p.y + o) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                         pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
        return;
    }
    for (int j = 0; j < 8 && k + j < p.w.K; ++j) {
        if (p.f32)
            ((float *)p.y)[o + j] = v[j];
        else
            ((__bf16 *)p.y)[o + j] = (__bf16)v[j];
    }
}

/*
 * A few rows times a packed matrix.  A workgroup of NW wavefronts owns 16 NT
 * rows of W and 16 MT rows of x; its wavefronts take the 128-wide chunks of K
 * in turn and add up in LDS at the end, so there is one launch and no scratch.
 *
 * v_mfma_f32_16x16x32_bf16 with x as the first operand and the weights as the
 * second: lane l holds column n = l % 16 and 8 consecutive k for the octet
 * q = l / 16, and gets sums of that same column, so a lane needs the scales
 * of one row of W alone.  A lane loads 16 bytes, the 32 codes of octets
 * 4q .. 4q + 3 of its row's chunk.
 *
 * MXFP4: the 32 codes are one block; the conversion to bf16 takes the block's
 * power of two along and stays exact.
 * INT: bf16 holds 16 + u exactly with u in its mantissa (0x4180 | u << 3), so
 * two shifted masks give two weights with no conversion, and
 *   sum_k x (u - z) = sum_k x (16 + u) - (16 + z) sum_k x.
 * The sum of x comes from a product with ones, in the same layout.  16 is the
 * smallest such offset; what the subtraction loses is under two bits of the
 * 32-bit sum.  Scales multiply the group's sum, so weights are never rounded.
 * For groups under 128 a 4 x 4 transpose among the lanes of a row (permlane
 * swaps) first brings octets 4j + q to lane q, so that product j covers the
 * 32 values from 32 j on, and each product lies within one group.
 */
template <bool MX, int GROUP, int MT, int NT, int NW, bool XVEC>
__global__ __launch_bounds__(NW * 64) void w4_gemm_kernel(W4GemmParams p)
{
    const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t c = lane & 15, q = lane >> 4;
    const int32_t n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
    const int32_t K = p.w.K, ng = p.w.ng;
    constexpr bool FLIP = !MX && GROUP < 128;      /* transposed octets        */
    constexpr int GC = MX ? 1 : 128 / GROUP;       /* groups a chunk           */

    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int32_t chunks = (K + 127) >> 7;
    for (int32_t ch = wave; ch < chunks; ch += NW) {
        const int32_t kc = ch << 7;
        uint4 raw[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int32_t n = n0 + 16 * t + c;
            raw[t] = make_uint4(0, 0, 0, 0);
            if (n < p.w.N && kc + 32 * q < K)
                raw[t] = *(const uint4 *)(p.w.codes + (int64_t)n * p.w.ldb + (kc >> 1) + 16 * q);
        }
        /* x: row m = lane % 16 of each row tile, 8 values for each of the
         * chunk's four products */
        bf16x8 xf[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int32_t m = m0 + 16 * i + c;
            const uint16_t *row = p.x + (int64_t)m * p.ldx;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t k = kc + (FLIP ? 32 * j + 8 * q : 32 * q + 8 * j);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (XVEC) {
                    if (m < p.M && k < K) v = *(const uint4 *)(row + k);
                } else if (m < p.M) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = k + e < K ? row[k + e] : 0u;
                    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
                }
                if constexpr (!MX) {
                    /* the codes' order: value i beside value i + 4 */
                    v = make_uint4((v.x & 0xFFFFu) | v.z << 16, v.x >> 16 | (v.z & 0xFFFF0000u),
                                   (v.y & 0xFFFFu) | v.w << 16, v.y >> 16 | (v.w & 0xFFFF0000u));
                }
                xf[i][j] = __builtin_bit_cast(bf16x8, v);
            }
        }
        if constexpr (MX) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int32_t n = n0 + 16 * t + c;
                uint32_t e = 127;
                if (n < p.w.N && kc + 32 * q < K) e = ((const uint8_t *)p.w.scales)[(int64_t)n * ng + (kc >> 5) + q];
                const float s = __builtin_bit_cast(float, e << 23);
                const uint32_t w[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bf16x2 b[4];
                    b[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0);
                    b[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1);
                    b[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2);
                    b[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3);
                    const bf16x8 wf = __builtin_bit_cast(bf16x8, b);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i][j], wf, acc[t][i], 0, 0, 0);
                }
            }
        } else {
            bf16x8 ones;
#pragma unroll
            for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;
            f32x4 sx[GC][MT];
#pragma unroll
            for (int g = 0; g < GC; ++g)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    sx[g][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 4 / GC; ++j)
                        sx[g][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i][g * (4 / GC) + j], ones, sx[g][i], 0, 0, 0);
                }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int32_t n = n0 + 16 * t + c;
                uint32_t w[4] = {raw[t].x, raw[t].y, raw[t].z, raw[t].w};
                if constexpr (FLIP) {
                    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                    auto d = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
                    auto f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
                    w[0] = d[0];
                    w[1] = d[1];
                    w[2] = f[0];
                    w[3] = f[1];
                }
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    float s = 0.0f, off = 24.0f;
                    if (n < p.w.N && kc + g * GROUP < K) {
                        const int64_t at = (int64_t)n * ng + kc / GROUP + g;
                        s = bf16_value(((const uint16_t *)p.w.scales)[at]);
                        if (p.w.zeros) off = 16.0f + (float)p.w.zeros[at];
                    }
                    f32x4 sum[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i) sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = g * (4 / GC); j < (g + 1) * (4 / GC); ++j) {
                        const uint4 b = make_uint4(((w[j] << 3) & 0x00780078u) | 0x41804180u, ((w[j] >> 1) & 0x00780078u) | 0x41804180u,
                                                   ((w[j] >> 5) & 0x00780078u) | 0x41804180u, ((w[j] >> 9) & 0x00780078u) | 0x41804180u);
                        const bf16x8 wf = __builtin_bit_cast(bf16x8, b);
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i][j], wf, sum[i], 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[t][i][r] += s * __builtin_fmaf(-off, sx[g][i][r], sum[i][r]);
                }
            }
        }
    }

    /* add the wavefronts' sums; entry (t, i, r, lane) is row 4 (lane / 16) + r,
     * column lane % 16 of its tile */
    constexpr int E = NT * MT * 4;
    __shared__ float red[NW][E][64];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][(t * MT + i) * 4 + r][lane] = acc[t][i][r];
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E * 64; e += NW * 64) {
        const int32_t el = e >> 6, ln = e & 63;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += red[w][el][ln];
        const int32_t t = el / (MT * 4), i = el / 4 % MT, r = el & 3;
        const int32_t m = m0 + 16 * i + 4 * (ln >> 4) + r, n = n0 + 16 * t + (ln & 15);
        if (m < p.M && n < p.w.N) {
            if (p.out_bf16)
                ((__bf16 *)p.y)[(int64_t)m * p.ldy + n] = (__bf16)sum;
            else
                ((float *)p.y)[(int64_t)m * p.ldy + n] = sum;
        }
    }
}

hipError_t launch_w4_quantize(const W4QuantParams &p, hipStream_t stream)
{
    const int64_t n = (int64_t)p.w.N * p.w.ng * (p.w.group >> 3);
    hipLaunchKernelGGL(w4_quantize_kernel, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_w4_dequantize(const W4QuantParams &p, hipStream_t stream)
{
    const int64_t n = (int64_t)p.w.N * ((p.w.K + 7) >> 3);
    hipLaunchKernelGGL(w4_dequantize_kernel, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

namespace {

template <bool MX, int GROUP, int MT, int NT, int NW>
void launch_one(const W4GemmParams &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)((p.w.N + 16 * NT - 1) / (16 * NT)), (uint32_t)((p.M + 16 * MT - 1) / (16 * MT)));
    if (p.xvec)
        hipLaunchKernelGGL((w4_gemm_kernel<MX, GROUP, MT, NT, NW, true>), grid, dim3(NW * 64), 0, stream, p);
    else
        hipLaunchKernelGGL((w4_gemm_kernel<MX, GROUP, MT, NT, NW, false>), grid, dim3(NW * 64), 0, stream, p);
}

template <bool MX, int GROUP>
void launch_rows(const W4GemmParams &p, int32_t cus, hipStream_t stream)
{
    (void)cus;
    if (p.M <= 16)
        launch_one<MX, GROUP, 1, 1, 8>(p, stream);
    else if (p.M <= 32)
        launch_one<MX, GROUP, 2, 2, 8>(p, stream);
    else
        launch_one<MX, GROUP, 4, 2, 4>(p, stream);
}

} /* namespace */

hipError_t launch_w4_gemm(const W4GemmParams &p, int32_t cus, hipStream_t stream)
{
    if (p.w.mx)
        launch_rows<true, 32>(p, cus, stream);
    else if (p.w.group == 32)
        launch_rows<false, 32>(p, cus, stream);
    else if (p.w.group == 64)
        launch_rows<false, 64>(p, cus, stream);
    else
        launch_rows<false, 128>(p, cus, stream);
    return hipGetLastError();
}

} /* namespace g355 */
