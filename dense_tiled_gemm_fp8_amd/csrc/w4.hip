/*
 * w4.hip -- matrices held in 4 bits with a scale for each group of K, and
 * products of a few bf16 rows with them.
 *
 *   INT    w[n][k] = (u[n][k] - z[n][g]) * s[n][g], u in 0..15, g = k / group,
 *          s bf16, z a byte (8 where there are no zero points)
 *   MXFP4  w[n][k] = e2m1(c[n][k]) * 2^(e[n][k / 32] - 127)
 *
 *   w4_quantize_kernel    8 consecutive elements a lane, the group's range by
 *                         shuffles among its group / 8 lanes
 *   w4_dequantize_kernel  8 consecutive elements a lane
 *   w4_gemm_kernel        y[m][n] = sum_k x[m][k] w[n][k]
 */
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "dma.h"
#include "serve.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

/* One octet (8 elements of a row) a thread.  Rows go by blockIdx.y where all of a
 * matrix's octets would not be counted in 31 bits.  (Four octets a thread, for
 * more loads in flight: 48.5 us against 43.6 for 8192 x 8192 bf16, 7.0 against 5.5
 * for 1000 x 3000 fp32; the dequantiser 26.4, 26.4 and 6.0, 4.8.) */
struct Octet {
    int32_t n, i;                 /* row, octet of the row                    */
    bool in;
};

__device__ __forceinline__ Octet octet(const W4QuantParams &p)
{
    Octet o;
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    const int32_t row = quotient((int32_t)id, p.by_row);
    o.i = (int32_t)id - row * p.per_row;
    const int64_t n = (int64_t)blockIdx.y * p.rows_y + row;
    o.in = row < p.rows_y && n < p.w.N;
    o.n = o.in ? (int32_t)n : 0;
    return o;
}

/* Value of the lane that CTRL names (a data-parallel-primitive control). */
template <int CTRL>
__device__ __forceinline__ float lane_move(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

/* Smallest and largest over LANES neighbours: swaps within pairs and fours,
 * then mirrored eights and sixteens (whose fours, eights agree by then). */
template <int LANES>
__device__ __forceinline__ void lane_range(float &lo, float &hi)
{
    lo = fminf(lo, lane_move<0xB1>(lo));
    hi = fmaxf(hi, lane_move<0xB1>(hi));
    lo = fminf(lo, lane_move<0x4E>(lo));
    hi = fmaxf(hi, lane_move<0x4E>(hi));
    if constexpr (LANES >= 8) {
        lo = fminf(lo, lane_move<0x141>(lo));
        hi = fmaxf(hi, lane_move<0x141>(hi));
    }
    if constexpr (LANES >= 16) {
        lo = fminf(lo, lane_move<0x140>(lo));
        hi = fmaxf(hi, lane_move<0x140>(hi));
    }
}

/* The group / 8 threads of a group are neighbours in a wavefront.
 *
 * w / s is rounded to nearest from the reciprocal r of s: q0 = w r is within an
 * ulp, and q0 + (w - q0 s) r is the quotient rounded to nearest (Markstein's
 * theorem; the residual is exact by the fused multiply-add).  A quotient that
 * would be subnormal rounds to the code of zero either way.
 *
 * Memory bounds it on large matrices: 8192 x 8192 bf16 to INT with groups of 64
 * moves 171 MB in 43.6 us, 3.9 TB/s, where a large copy reaches 4.8.  On small
 * ones the chain of a load, the range and a store does: 1000 x 3000 fp32 to MXFP4,
 * 14 MB, in 5.2 us. */
template <bool MX, int LANES>
__global__ __launch_bounds__(256) void w4_quantize_kernel(W4QuantParams p)
{
    constexpr int LOG2 = LANES == 4 ? 2 : LANES == 8 ? 3 : 4;
    const Octet o = octet(p);
    float v[8];
    if (o.in) {
        load8_row(p, o.n, o.i * 8, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, v[j]);
        hi = fmaxf(hi, v[j]);
    }
    lane_range<LANES>(lo, hi);
    const int32_t kk = o.i * 8;
    if (!o.in || kk >= p.w.K) return;
    const int64_t at = (int64_t)o.n * p.w.ng + (o.i >> LOG2);
    const bool first = (o.i & (LANES - 1)) == 0;
    uint32_t word = 0;
    if constexpr (MX) {
        const uint32_t bits = __builtin_bit_cast(uint32_t, fmaxf(-lo, hi));
        /* exponent of the largest less 2, not under 2^-127 (its exponent
         * field counts from 127; a subnormal is under 2^-126) */
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
        const float r = 1.0f / s;
        auto quotient = [&](float w) __attribute__((always_inline)) {
            const float q0 = w * r;
            return __builtin_fmaf(__builtin_fmaf(-q0, s, w), r, q0);
        };
        float z = 8.0f;
        if (p.w.zeros) z = fminf(fmaxf(rintf(quotient(-lo)), 0.0f), 15.0f);
        if (first) {
            ((__bf16 *)p.w.scales)[at] = (__bf16)s;
            if (p.w.zeros) p.w.zeros[at] = (uint8_t)z;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = fminf(fmaxf(rintf(quotient(v[j])) + z, 0.0f), 15.0f);
            word |= (uint32_t)u << (4 * j);
        }
        /* elements past K read as zero, whose code is z */
        if (kk + 8 > p.w.K) word &= (1u << (4 * (p.w.K - kk))) - 1u;
    }
    *(uint32_t *)(p.w.codes + (int64_t)o.n * p.w.ldb + (kk >> 1)) = word;
}

/* 8 weights a lane from one dword of codes and their group's scale; exact in fp32
 * (a code less a zero point has 9 bits, a scale 8), rounded once for bf16.  The
 * store bounds it: 8192 x 8192 INT to bf16, 171 MB in 26 us, 6.6 TB/s, right after
 * the quantiser (codes still in the caches), 37.9 us, 4.5 TB/s, with other
 * matrices between; to fp32, 305 MB, 61.9 us, 4.9 TB/s.  1000 x 3000 MXFP4 to bf16
 * 4.0 us, 7.6 MB, to fp32 5.4 us, 13.6 MB: the chain of a load and a store. */
__global__ __launch_bounds__(256) void w4_dequantize_kernel(W4QuantParams p)
{
    const Octet o = octet(p);
    if (!o.in) return;
    const int32_t group_log2 = p.w.group == 32 ? 2 : p.w.group == 64 ? 3 : 4;   /* in octets */
    const uint32_t word = *(const uint32_t *)(p.w.codes + (int64_t)o.n * p.w.ldb + o.i * 4);
    const int64_t in_group = (int64_t)o.n * p.w.ng + (o.i >> group_log2);
    const uint32_t scale = p.w.mx ? ((const uint8_t *)p.w.scales)[in_group] : ((const uint16_t *)p.w.scales)[in_group];
    const uint32_t zero = p.w.zeros ? p.w.zeros[in_group] : 8;
    const int32_t kk = o.i * 8;
    float v[8];
    if (p.w.mx) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = (word >> (4 * j)) & 15u, m = c & 7u;
            /* magnitude codes 0 and 1 are 0 and 0.5, the others (2 + m % 2)
             * times 2^(m / 2 - 2) */
            const float mag = m < 2 ? 0.5f * (float)m : __builtin_ldexpf((float)(2 + (m & 1u)), (int)(m >> 1) - 2);
            v[j] = scale == 255 ? __builtin_nanf("") : __builtin_ldexpf(c & 8u ? -mag : mag, (int)scale - 127);
        }
    } else {
        const float s = bf16_value(scale), z = (float)zero;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((float)((word >> (4 * j)) & 15u) - z) * s;
    }
    const int64_t at = (int64_t)o.n * p.ld + kk;
    if (p.vec && kk + 8 <= p.w.K) {
        if (p.f32) {
            *(float4 *)((float *)p.y + at) = make_float4(v[0], v[1], v[2], v[3]);
            *(float4 *)((float *)p.y + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *(uint4 *)((uint16_t *)p.y + at) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
        return;
    }
    for (int j = 0; j < 8 && kk + j < p.w.K; ++j) {
        if (p.f32)
            ((float *)p.y)[at + j] = v[j];
        else
            ((__bf16 *)p.y)[at + j] = (__bf16)v[j];
    }
}

/* Weights of a dword of codes, in bf16 and in the order that x is put into:
 * MXFP4 in the codes' order, times the block's power of two; INT 0 2, 4 6,
 * 1 3, 5 7, as whole numbers.  A byte u = 0 .. 15 read as E4M3 is u * 2^-9
 * (subnormals and the first binade are one arithmetic sequence), so masked
 * nibbles convert in pairs: 7 instructions for 8 weights, where shifting each
 * nibble into a bf16 significand takes 8 and leaves an offset to take off. */
template <bool MX>
__device__ __forceinline__ bf16x8 decode_codes(uint32_t w, float s)
{
    bf16x2 b[4];
    if constexpr (MX) {
        b[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
        b[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
        b[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
        b[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    } else {
        const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
        b[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
        b[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
        b[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
        b[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    }
    return __builtin_bit_cast(bf16x8, b);
}

template <bool MX>
__device__ __forceinline__ bf16x8 order_x(u32x4 v)
{
    if constexpr (!MX)
        v = u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
                  __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
    return __builtin_bit_cast(bf16x8, v);
}

/* 4 x 4 transpose of dwords among the four lanes of a row (lane / 16): lane q
 * gets dword q of all four. */
__device__ __forceinline__ void transpose4(uint32_t (&w)[4])
{
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w[0] = d[0];
    w[1] = d[1];
    w[2] = f[0];
    w[3] = f[1];
}

__device__ __forceinline__ bf16x8 ones8()
{
    return __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
}

/* The wavefronts' sums, added in order and stored: entry (t, i, r, lane) is
 * row m0 + 16 i + 4 (lane / 16) + r (R = 1: m0 + lane / 16), column
 * n0 + 16 t + lane % 16. */
template <int NT, int RT, int R, int NW>
__device__ __forceinline__ void store_sums(const W4GemmParams &p, float *store, int32_t wave, int32_t lane, int32_t m0, int32_t n0,
                                           const f32x4 (&acc)[NT][RT])
{
    constexpr int E = NT * RT * R;
    float(*red)[E][64] = (float(*)[E][64])store;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) red[wave][(t * RT + i) * R + r][lane] = acc[t][i][r];
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E * 64; e += NW * 64) {
        const int32_t el = e >> 6, ln = e & 63;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += red[w][el][ln];
        const int32_t t = el / (RT * R), i = el / R % RT, r = el % R;
        const int32_t m = m0 + 16 * i + (R == 4 ? 4 * (ln >> 4) + r : ln >> 4), n = n0 + 16 * t + (ln & 15);
        if (m < p.M && n < p.w.N) {
            if (p.out_bf16)
                ((__bf16 *)p.y)[(int64_t)m * p.ldy + n] = (__bf16)sum;
            else
                ((float *)p.y)[(int64_t)m * p.ldy + n] = sum;
        }
    }
}

/*
 * A few rows times a packed matrix.  A workgroup of NW wavefronts owns 16 NT
 * rows of W and up to 16 MT rows of x; its wavefronts take a run of the
 * 128-wide chunks of K each and add up in LDS at the end, so there is one
 * launch, no scratch, and each code is read once for 16 MT rows.
 *
 * v_mfma_f32_16x16x32_bf16 with x as the first operand and the weights as the
 * second: lane l holds column n = l % 16 and 8 consecutive k for the octet
 * q = l / 16, and gets sums of that same column, so a lane needs the scales
 * of one row of W alone.  A lane takes 16 bytes, the 32 codes of octets
 * 4q .. 4q + 3 of its row's chunk.
 *
 * MXFP4: the 32 codes are one block; the conversion to bf16 takes the block's
 * power of two along and stays exact.
 * INT: sum_k x (u - z) = sum_k x u - z sum_k x; the sum of x comes from a
 * product with ones, in the same layout.  Scales multiply the group's sum, so
 * weights are never rounded.  For groups under 128 a transpose among the lanes
 * of a row first brings octets 4j + q to lane q, so that product j covers the
 * 32 values from 32 j on, and each product lies within one group.
 *
 * The vector memory unit takes four lanes at a time and wants their 64 bytes
 * contiguous; the matrix instruction wants consecutive lanes in different
 * rows.  So copies go straight to LDS with lanes along rows (four lanes a row
 * of a chunk's codes, 16 a row of x) and each wavefront reads its own copies
 * back in the matrix order.  The 16-byte units of a row are exchanged by row
 * number, which leaves the reads free of bank conflicts.  Loads in the matrix
 * order took 64 cycles each instead of 16 (one token against 16384 x 8192: 45 us
 * with them, 20 with the copies).
 *
 * A wavefront has up to four chunks in LDS, one read while the others arrive; it
 * waits for its own copies alone, so there is no barrier in the loop.
 *
 * Rows of x past M and of W past N are read as the last ones (their sums are
 * not stored), which leaves the loop without masks.  MT = 0 is for M <= 4: row
 * m sits in row 4m of the instruction's 16, so a lane scales one sum, not four.
 *
 * ODD = false: K is a multiple of 128, rows are 16-byte aligned, scales and zero
 * points fill whole dwords.  ODD = true: any K of 8 or more and any alignment of
 * rows, scales and zero points (the copies take any byte address).  What a chunk
 * has past K reads as zero: whole units by an offset out of range, the unit of x
 * that K ends in by a shift in LDS.  Scales and zero points of a dword that would
 * pass its array's end are read from further down and shifted.  One token against
 * 16000 x 8000 takes 19.2 us (16000 x 8064, even: 15.7; a chunk of 8000's rows lies
 * across two lines), 32 against 8000 x 7999 17.1, where operands loaded in the
 * matrix order took 192.
 *
 * Measured: one token against 16384 x 8192 INT (groups of 64, zero points), 73 MB:
 * 15.5 us with three matrices in turn, 4.74 TB/s, what a large copy reaches, but
 * those fit in the 256 MB cache before memory: 19.8 us, 3.7 TB/s, with eleven.
 * 1024 x 1024: 2.6 us, the latency of one round of copies, sums and a join (5 rows
 * against 3000 x 777 INT 3.7).  32 tokens against 8192 x 8192 MXFP4: 11.8 us with
 * three matrices in turn, 15.7 with 18; every workgroup of 32 rows of W reads all
 * of x, 134 MB from the L2 beside 37 MB of codes, and x takes 8 of a chunk's 10 KB
 * in LDS, so fewer bytes are in flight.  INT at 32 tokens 19.5, at 64 tokens 31.5
 * (MXFP4 21.7): there a chunk is 16 KB of x and 2 of codes, of which a wavefront
 * has room for two.
 */
template <bool MX, int GROUP, bool ZEROS, int MT, int NT, int NW, bool ODD>
__global__ __launch_bounds__(NW * 64) void w4_gemm_kernel(W4GemmParams p)
{
    constexpr int RT = MT ? MT : 1;                /* row tiles                */
    constexpr int R = MT ? 4 : 1;                  /* sums of a tile in a lane */
    constexpr bool FLIP = !MX && GROUP < 128;      /* transposed octets        */
    constexpr int GC = MX ? 1 : 128 / GROUP;       /* groups a chunk           */
    constexpr int XL = MT ? 4 * MT : 1;            /* copies of x a chunk      */
    constexpr int SD = GC == 4 ? 2 : 1;            /* dwords of scales a row   */
    constexpr int COPIES = NT + XL;                /* of a chunk               */
    constexpr int SLOT = COPIES * 1024;
    constexpr int QUAD = NT * (SD + ZEROS) * 256;  /* scales of four chunks    */
    constexpr int FIT = ((MT ? 163840 : 81920) / NW - 2 * QUAD) / SLOT, DEPTH = FIT < 4 ? FIT : 4;
    constexpr int OWN = DEPTH * SLOT + 2 * QUAD;
    static_assert(NT * RT * R * 256 <= OWN && DEPTH >= 2 && COPIES * (DEPTH - 1) < 64, "LDS and waits");
    const int32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t c = lane & 15, q = lane >> 4;
    const int32_t n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * RT);
    const int32_t K = p.w.K, ng = p.w.ng;

    /* per-lane offsets from the workgroup's first rows (64 rows stay under
     * 2^31 bytes: rows are at most 2^23 elements apart) */
    const int32_t lrow = lane >> 2, lpiece = (lane & 3) ^ (lrow >> 2);
    uint32_t code_at[NT], x_at[XL];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        code_at[t] = (uint32_t)((min(n0 + 16 * t + lrow, p.w.N - 1) - n0) * (int32_t)p.w.ldb + 16 * lpiece);
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int32_t row = 4 * i + (lane >> 4);
        x_at[i] = (uint32_t)((min(m0 + row, p.M - 1) - m0) * (int32_t)p.ldx + 8 * ((lane & 15) ^ (row & 15))) * 2;
    }
    const i32x4 rc = rsrc_words(p.w.codes + (int64_t)n0 * p.w.ldb);
    /* ODD: a dword further down, as the last one may begin before row n0 */
    const int32_t lead = ODD && n0 > 0 ? 4 : 0;
    const i32x4 rs = rsrc_words((const uint8_t *)p.w.scales + ((int64_t)n0 * ng * (MX ? 1 : 2) - lead));
    const i32x4 rz = rsrc_words(ZEROS ? p.w.zeros + ((int64_t)n0 * ng - lead) : p.w.codes);
    const i32x4 rx = rsrc_words(p.x + (int64_t)m0 * p.ldx);

    /* last byte offsets that a dword of scales or zero points may be read from */
    int32_t last_scale = 0, last_zero = 0;
    if constexpr (ODD) {
        const int64_t left = (int64_t)(p.w.N - n0) * ng;
        last_scale = (int32_t)min(left * (MX ? 1 : 2) - 4 + lead, (int64_t)0x40000000);
        last_zero = (int32_t)min(left - 4 + lead, (int64_t)0x40000000);
    }

    __shared__ __align__(16) uint8_t store[NW * OWN];
    const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(store) + wave * OWN);
    const uint8_t *own = store + wave * OWN;

    /* A wavefront takes a run of chunks, so that its copies in flight are
     * neighbours in memory, and begins it at a place of the workgroup's own, so
     * that workgroups spread over the memory channels: rows are often a power
     * of two apart. */
    const int32_t chunks = ODD ? (K + 127) >> 7 : K >> 7;
    const int32_t first = chunks * wave / NW;
    const int32_t count = chunks * (wave + 1) / NW - first;
    const int32_t start = (int32_t)__umulhi(blockIdx.x * p.spread, (uint32_t)count);
    auto chunk = [&](int32_t i) __attribute__((always_inline)) {
        const int32_t ch = i + start;
        return first + (ch >= count ? ch - count : ch);
    };

    /* A chunk's copies into a slot; past the last chunk they read nothing. */
    auto copy = [&](int32_t slot, int32_t i) __attribute__((always_inline)) {
        const uint32_t at = base + (uint32_t)slot * SLOT;
        const uint32_t ch = (uint32_t)chunk(i), kb = i < count ? ch << 6 : kOOB, kx = i < count ? ch << 8 : kOOB;
        if constexpr (ODD) {
            if ((int32_t)ch == chunks - 1 && i < count) {
                /* K ends in this chunk: units past it read nothing, and the
                 * one of x that it ends in is read up to K, eight elements
                 * that the wait below shifts to their place */
                const int32_t left = K - ((int32_t)ch << 7);
                const uint32_t cb = 32 * lpiece < left ? kb : kOOB;
                unroll<NT>([&](auto t) { dma16<t * 1024>(rc, at, code_at[t] + cb); });
                unroll<XL>([&](auto i) {
                    const int32_t k = 8 * ((lane & 15) ^ ((4 * i + (lane >> 4)) & 15));
                    const uint32_t xb = k >= left ? kOOB : kx - 2 * (uint32_t)max(k + 8 - left, 0);
                    dma16<(NT + i) * 1024>(rx, at, x_at[i] + xb);
                });
                return;
            }
        }
        unroll<NT>([&](auto t) { dma16<t * 1024>(rc, at, code_at[t] + kb); });
        unroll<XL>([&](auto i) { dma16<(NT + i) * 1024>(rx, at, x_at[i] + kx); });
    };
    /* Scales of the run's chunks i .. i + 3 (the last again past its end): lane
     * 4r + d copies row r's of chunk i + d.  Rows are far apart, so each of
     * these copies touches 16 lines for a few bytes of each; by fours they
     * touch a quarter as many. */
    auto copy_scales = [&](int32_t half, int32_t i) __attribute__((always_inline)) {
        const uint32_t at = base + DEPTH * SLOT + (uint32_t)half * QUAD;
        const int32_t ch = chunk(min(i + (lane & 3), count - 1));
        unroll<NT>([&](auto t) {
            const uint32_t si = (uint32_t)((min(n0 + 16 * t + lrow, p.w.N - 1) - n0) * ng + ch * (MX ? 4 : GC));
            if constexpr (ODD) {
                /* any byte address, and never past the array's end */
                constexpr int PER = (SD + ZEROS) * 256;
                const int32_t byte = (int32_t)(MX ? si : 2 * si) + lead;
                dma4(rs, at + t * PER, (uint32_t)min(byte, last_scale));
                if constexpr (SD == 2) dma4(rs, at + t * PER + 256, (uint32_t)min(byte + 4, last_scale));
                if constexpr (ZEROS) dma4(rz, at + t * PER + SD * 256, (uint32_t)min((int32_t)si + lead, last_zero));
                return;
            }
            const uint32_t ks = MX ? si : 2 * si & ~3u;
            constexpr int PER = (SD + ZEROS) * 256;
            dma4(rs, at + t * PER, ks);
            if constexpr (SD == 2) dma4(rs, at + t * PER + 256, ks + 4);
            if constexpr (ZEROS) dma4(rz, at + t * PER + SD * 256, si & ~3u);
        });
    };

    f32x4 acc[NT][RT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int32_t code_get = c * 64 + ((q ^ (c >> 2)) << 4);
    const int32_t xrow = MT ? c : c >> 2;
    if (count > 0) {
        copy_scales(0, 0);
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d) copy(d, d);
    }
    int32_t slot = 0, free_slot = DEPTH - 1;
#pragma unroll 1
    for (int32_t i = 0; i < count; ++i) {
        /* the slot to fill is the one read in the step before: those reads
         * have returned */
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if ((i & 3) == 0 && i + 4 < count) copy_scales((i >> 2 & 1) ^ 1, i + 4);
        copy(free_slot, i + DEPTH - 1);
        /* all but the copies of the next DEPTH - 1 chunks: this chunk's, and
         * scales sent off four steps ago */
        wait_vmcnt<(DEPTH - 1) * COPIES>();
        const uint8_t *in = own + slot * SLOT, *xin = in + NT * 1024;
        const uint8_t *sin = own + DEPTH * SLOT + (i >> 2 & 1) * QUAD + 4 * (4 * c + (i & 3));
        const int32_t ch = chunk(i);
        const int32_t left = K - (ch << 7);            /* of K, from this chunk on */
        if constexpr (ODD) {
            if (left < 128 && (left & 7) != 0) {
                constexpr int ROWS = MT ? 16 * MT : 4;
                if (lane < ROWS) {
                    uint16_t *at = (uint16_t *)(own + slot * SLOT + NT * 1024 + lane * 256 + (((left >> 3) ^ (lane & 15)) << 4));
                    const int32_t by = 8 - (left & 7);
                    uint16_t e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = j + by < 8 ? at[j + by] : (uint16_t)0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) at[j] = e[j];
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
        uint32_t w[NT][4], sc[NT][SD], zp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const u32x4 v = *(const u32x4 *)(in + t * 1024 + code_get);
            w[t][0] = v[0];
            w[t][1] = v[1];
            w[t][2] = v[2];
            w[t][3] = v[3];
            if constexpr (FLIP) transpose4(w[t]);
            const int32_t row = 16 * t + c;
            zp[t] = 0x08080808u;
            const uint8_t *st = sin + t * ((SD + ZEROS) * 256);
            sc[t][0] = *(const uint32_t *)st;
            if constexpr (SD == 2) sc[t][1] = *(const uint32_t *)(st + 256);
            if constexpr (ZEROS) zp[t] = *(const uint32_t *)(st + SD * 256);
            if constexpr (ODD) {
                /* read from further down at the array's end */
                const int32_t si = (min(n0 + row, p.w.N - 1) - n0) * ng + ch * (MX ? 4 : GC), byte = (MX ? si : 2 * si) + lead;
                sc[t][0] >>= 8 * min(max(byte - last_scale, 0), 3);
                if constexpr (SD == 2) sc[t][1] >>= 8 * min(max(byte + 4 - last_scale, 0), 3);
                if constexpr (ZEROS) zp[t] >>= 8 * min(max(si + lead - last_zero, 0), 3);
                if constexpr (MX) {
                    /* codes past K are zeros, of a block past it the scale 1:
                     * others might be infinities */
                    sc[t][0] = 32 * q < left ? sc[t][0] >> (8 * q) & 0xFFu : 127u;
                    if (left < 128)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int32_t n = left - 32 * q - 8 * j;
                            if (n < 8) w[t][j] &= n > 0 ? (1u << (4 * n)) - 1u : 0u;
                        }
                }
            } else if constexpr (MX) {
                sc[t][0] = sc[t][0] >> (8 * q) & 0xFFu;
            } else if constexpr (GC < 4) {
                /* the dword may begin before this chunk's part of it */
                const uint32_t at = (uint32_t)((min(n0 + row, p.w.N - 1) - n0) * ng + ch * GC);
                if constexpr (GC == 1) sc[t][0] >>= 16 * (at & 1);
                if constexpr (ZEROS) zp[t] >>= 8 * (at & 3);
            }
        }
        f32x4 sum[NT][RT], sx[RT];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!MX && j % (4 / GC) == 0) {
#pragma unroll
                for (int i2 = 0; i2 < RT; ++i2) {
                    sx[i2] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = 0; t < NT; ++t) sum[t][i2] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
            }
            bf16x8 xf[RT];
#pragma unroll
            for (int i2 = 0; i2 < RT; ++i2) {
                xf[i2] = order_x<MX>(*(const u32x4 *)(xin + (16 * i2 + xrow) * 256 + (((FLIP ? 4 * j + q : 4 * q + j) ^ xrow) << 4)));
                if constexpr (!MX) sx[i2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i2], ones8(), sx[i2], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bf16x8 wf = decode_codes<MX>(w[t][j], __builtin_bit_cast(float, sc[t][0] << 23));
#pragma unroll
                for (int i2 = 0; i2 < RT; ++i2) {
                    if constexpr (MX)
                        acc[t][i2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i2], wf, acc[t][i2], 0, 0, 0);
                    else
                        sum[t][i2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i2], wf, sum[t][i2], 0, 0, 0);
                }
            }
            if (!MX && j % (4 / GC) == 4 / GC - 1) {
                const int g = j / (4 / GC);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t two = sc[t][g >> 1];
                    float s = __builtin_bit_cast(float, g & 1 ? two & 0xFFFF0000u : two << 16);
                    if (ODD && g * GROUP >= left) s = 0.0f;        /* a group past K */
                    const float z = (float)((zp[t] >> (8 * g)) & 0xFFu);
#pragma unroll
                    for (int i2 = 0; i2 < RT; ++i2)
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[t][i2][r] += s * __builtin_fmaf(-z, sx[i2][r], sum[t][i2][r]);
                }
            }
        }
        free_slot = slot;
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
    wait_vmcnt<0>();                               /* copies that read nothing */
    __syncthreads();
    store_sums<NT, RT, R, NW>(p, (float *)store, wave, lane, m0, n0, acc);
}

/* The same product for what the kernel above does not take (K under 8, scales or
 * zero points of less than a dword in all): 16 rows of W and of x a workgroup,
 * operands loaded in the matrix order, elements past K read as zero.  Nothing to
 * gain there: the launch is all it takes. */
constexpr int kW4AnyWaves = 8;

template <bool MX, int GROUP>
__global__ __launch_bounds__(kW4AnyWaves * 64) void w4_gemm_any_kernel(W4GemmParams p)
{
    constexpr bool FLIP = !MX && GROUP < 128;
    constexpr int GC = MX ? 1 : 128 / GROUP;
    const int32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t c = lane & 15, q = lane >> 4;
    const int32_t n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
    const int32_t K = p.w.K, n = min(n0 + c, p.w.N - 1), m = min(m0 + c, p.M - 1);
    const uint8_t *row = p.w.codes + (int64_t)n * p.w.ldb;
    const uint16_t *x = p.x + (int64_t)m * p.ldx;
    const int64_t g0 = (int64_t)n * p.w.ng;
    __shared__ float store[kW4AnyWaves * 4 * 64];

    f32x4 acc[1][1];
    acc[0][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t kc = wave << 7; kc < K; kc += kW4AnyWaves << 7) {
        u32x4 raw = {0, 0, 0, 0};
        if (kc + 32 * q < K) raw = *(const u32x4 *)(row + (kc >> 1) + 16 * q);
        uint32_t w[4] = {raw[0], raw[1], raw[2], raw[3]};
        if constexpr (FLIP) transpose4(w);
        bf16x8 xf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t k = kc + (FLIP ? 32 * j + 8 * q : 32 * q + 8 * j);
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = k + e < K ? x[k + e] : 0u;
            xf[j] = order_x<MX>(u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16});
        }
        if constexpr (MX) {
            const uint32_t e = kc + 32 * q < K ? ((const uint8_t *)p.w.scales)[g0 + (kc >> 5) + q] : 127u;
            /* codes past K are zeros: with a scale of 2^126 others might be
             * infinities, which x = 0 does not keep out of the sums */
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t left = K - kc - 32 * q - 8 * j;
                if (left < 8) w[j] &= left > 0 ? (1u << (4 * left)) - 1u : 0u;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[0][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j], decode_codes<MX>(w[j], __builtin_bit_cast(float, e << 23)),
                                                                    acc[0][0], 0, 0, 0);
        } else {
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float s = 0.0f, z = 8.0f;
                if (kc + g * GROUP < K) {
                    const int64_t at = g0 + kc / GROUP + g;
                    s = bf16_value(((const uint16_t *)p.w.scales)[at]);
                    if (p.w.zeros) z = (float)p.w.zeros[at];
                }
                f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f}, sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = g * (4 / GC); j < (g + 1) * (4 / GC); ++j) {
                    sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j], ones8(), sx, 0, 0, 0);
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j], decode_codes<MX>(w[j], 0.0f), sum, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[0][0][r] += s * __builtin_fmaf(-z, sx[r], sum[r]);
            }
        }
    }
    store_sums<1, 1, 4, kW4AnyWaves>(p, store, wave, lane, m0, n0, acc);
}

namespace {

/* Rows of `per_row` octets over the grid. */
dim3 octet_grid(W4QuantParams &p, int64_t per_row)
{
    p.per_row = (int32_t)per_row;
    p.by_row = divider(per_row);
    p.rows_y = (int32_t)std::min<int64_t>(p.w.N, std::max<int64_t>(1, (((int64_t)1 << 31) - 256) / per_row));
    return dim3((uint32_t)((p.rows_y * per_row + 255) / 256), (uint32_t)((p.w.N + p.rows_y - 1) / p.rows_y));
}

template <bool MX, int LANES>
void launch_quantize_group(W4QuantParams &p, hipStream_t stream)
{
    const dim3 grid = octet_grid(p, (int64_t)p.w.ng * LANES);
    hipLaunchKernelGGL((w4_quantize_kernel<MX, LANES>), grid, dim3(256), 0, stream, p);
}

} /* namespace */

hipError_t launch_w4_quantize(const W4QuantParams &p0, hipStream_t stream)
{
    W4QuantParams p = p0;
    if (p.w.mx)
        launch_quantize_group<true, 4>(p, stream);
    else if (p.w.group == 32)
        launch_quantize_group<false, 4>(p, stream);
    else if (p.w.group == 64)
        launch_quantize_group<false, 8>(p, stream);
    else
        launch_quantize_group<false, 16>(p, stream);
    return hipGetLastError();
}

hipError_t launch_w4_dequantize(const W4QuantParams &p0, hipStream_t stream)
{
    W4QuantParams p = p0;
    const dim3 grid = octet_grid(p, ((int64_t)p.w.K + 7) >> 3);
    hipLaunchKernelGGL(w4_dequantize_kernel, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

namespace {

template <bool MX, int GROUP, bool ZEROS, int MT, int NT, int NW>
void launch_one(const W4GemmParams &p, hipStream_t stream)
{
    const int32_t rows = MT ? 16 * MT : 16;
    const dim3 grid((uint32_t)((p.w.N + 16 * NT - 1) / (16 * NT)), (uint32_t)((p.M + rows - 1) / rows));
    W4GemmParams q = p;
    q.spread = (uint32_t)(0xFFFFFFFFu / grid.x);
    if (p.even)
        hipLaunchKernelGGL((w4_gemm_kernel<MX, GROUP, ZEROS, MT, NT, NW, false>), grid, dim3(NW * 64), 0, stream, q);
    else
        hipLaunchKernelGGL((w4_gemm_kernel<MX, GROUP, ZEROS, MT, NT, NW, true>), grid, dim3(NW * 64), 0, stream, q);
}

/* Rows of W a workgroup (16 NT): more of them read x less often, fewer of them
 * make more workgroups, and one a compute unit is wanted (the device has 256): 16
 * rows up to N = 4096, 32 up to 8192, 64 beyond (32 for M <= 4 and M > 32).  us,
 * INT with groups of 64 and zero points / MXFP4, 14 to 40 matrices in turn:
 *   M = 1:  N 4096, K 4096   NT 1: 5.1 / 4.2,    2: 5.7 / 4.5
 *           N 8000, K 8064   NT 1: 13.1 / 9.8,   2: 10.6 / 9.4
 *   M = 8:  N 5120, K 5120   NT 1: 10.2 / 8.4,   2: 8.1 / 6.5
 *           N 8192, K 8192   NT 2: 14.4 / 11.4,  4: 20.3 / 15.7
 *           N 9216, K 4096   NT 2: 12.5 / 9.7,   4: 11.4 / 7.9
 *   M = 32: N 4096, K 4096   NT 1: 8.7 / 6.7,    2: 10.3 / 7.2
 *           N 8000, K 8064   NT 1: 27.6 / 24.8,  2: 19.4 / 17.2
 *           N 8192, K 8192   NT 2: 19.4 / 15.7,  4: 27.6 / 20.4
 *           N 9216, K 4096   NT 2: 20.0 / 13.4,  4: 16.5 / 11.4
 *   M = 64: N 4096, K 4096   NT 1: 13.1 / 9.3,   2: 16.4 / 10.0
 *           N 8000, K 8064   NT 1: 42.3 / 36.8,  2: 31.8 / 24.0 */
template <bool MX, int GROUP, bool ZEROS>
void launch_rows(const W4GemmParams &p, hipStream_t stream)
{
    const bool few = p.w.N <= 4096, many = p.w.N > 8192;
    if (p.tiny) {
        const dim3 grid((uint32_t)((p.w.N + 15) / 16), (uint32_t)((p.M + 15) / 16));
        hipLaunchKernelGGL((w4_gemm_any_kernel<MX, GROUP>), grid, dim3(kW4AnyWaves * 64), 0, stream, p);
    } else if (p.M <= 4) {
        if (few)
            launch_one<MX, GROUP, ZEROS, 0, 1, 8>(p, stream);
        else
            launch_one<MX, GROUP, ZEROS, 0, 2, 8>(p, stream);
    } else if (p.M <= 16) {
        if (few)
            launch_one<MX, GROUP, ZEROS, 1, 1, 8>(p, stream);
        else if (!many)
            launch_one<MX, GROUP, ZEROS, 1, 2, 8>(p, stream);
        else
            launch_one<MX, GROUP, ZEROS, 1, 4, 4>(p, stream);
    } else if (p.M <= 32) {
        if (few)
            launch_one<MX, GROUP, ZEROS, 2, 1, 4>(p, stream);
        else if (!many)
            launch_one<MX, GROUP, ZEROS, 2, 2, 4>(p, stream);
        else
            launch_one<MX, GROUP, ZEROS, 2, 4, 4>(p, stream);
    } else {
        if (few)
            launch_one<MX, GROUP, ZEROS, 4, 1, 4>(p, stream);
        else
            launch_one<MX, GROUP, ZEROS, 4, 2, 4>(p, stream);
    }
}

} /* namespace */

hipError_t launch_w4_gemm(const W4GemmParams &p, hipStream_t stream)
{
    if (p.w.mx)
        launch_rows<true, 32, false>(p, stream);
    else if (p.w.group == 32)
        p.w.zeros ? launch_rows<false, 32, true>(p, stream) : launch_rows<false, 32, false>(p, stream);
    else if (p.w.group == 64)
        p.w.zeros ? launch_rows<false, 64, true>(p, stream) : launch_rows<false, 64, false>(p, stream);
    else
        p.w.zeros ? launch_rows<false, 128, true>(p, stream) : launch_rows<false, 128, false>(p, stream);
    return hipGetLastError();
}

} /* namespace g355 */
