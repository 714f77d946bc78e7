/*
 * block.hip -- products of E4M3 matrices that hold an fp32 scale for each block of
 * 128 K-values (x: of a row, w: of 128 rows), one or two at a time:
 *
 *   p_w[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in b} x[m][k] w[n][k]
 *   y = p_w,  or  y = act(p_gate) p_up
 *
 * A block's inner sum comes from the matrix instruction over 128 K-values begun at
 * zero, and one fused multiply-add takes it, times the product of its two scales,
 * into the fp32 sum.  Weights are the instruction's first operand and tokens the
 * second, so that a lane's sums are of one token: its scale is one register, and
 * the weights' scale is one for all.
 *
 * The 8-bit instruction sums products in groups of 8 K-values, each product cut
 * off at 2^-13 of the largest of its group (measured: 1 + 2^-13 within a group of
 * 8 is exact, 1 + 2^-14 is 1, and between groups 24 bits are kept).  Against normal
 * data that is 3e-4 of the result's size: a sixth of bf16's rounding, which it is
 * used for.  Rows of fp32, and codes whose scales are fp32, are made from sums of 32
 * bits: for them (EXACT) the codes of x and w become bf16, which holds them exactly,
 * and the 16-bit instruction sums them in fp32 at half the rate (4096 x 4096x4096:
 * rows of bf16 67 us, of fp32 126).
 *
 *   block_rows_kernel    up to 64 tokens: the stream of weights counts, K split among
 *                        wavefronts
 *   block_stream_kernel  some 128 tokens: the same, with wavefronts that only copy
 *   block_tile_kernel    many tokens: the matrix units count
 *   block_finish_kernel  joins parts of K, activates, quantises
 */
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "block.h"
#include "dma.h"
#include "sched.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ int lane_id()
{
    return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
}

/* 8 codes as bf16: dwords 2 j and 2 j + 1 of a fragment. */
__device__ __forceinline__ bf16x8 widen(const i32x8 &f, int j)
{
    const int lo = f[2 * j], hi = f[2 * j + 1];
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

/* act(g) u.  GELU (tanh): 0.5 g (1 + tanh z) = g / (1 + exp(-2 z)). */
__device__ __forceinline__ float gated(float g, float u, int32_t act)
{
    const float z = act == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.0f + __expf(-z)) * u;
}

/* Memory takes vectors at any address of whole elements. */
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

/* Four sums of consecutive columns from n on, as rows of y. */
__device__ __forceinline__ void store4(const BlockGemmParams &p, int32_t m, int32_t n, const f32x4 &v)
{
    const int64_t at = (int64_t)m * p.ldy + n;
    const float a = v[0], b = v[1], c = v[2], d = v[3];
    if (n + 4 <= p.N) {
        if (p.y_f32)
            *(f32x4_any *)((float *)p.y + at) = f32x4_any{a, b, c, d};
        else
            *(u32x2_any *)((uint16_t *)p.y + at) = u32x2_any{pack_bf16(a, b), pack_bf16(c, d)};
        return;
    }
    const float e[4] = {a, b, c, d};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= p.N) continue;
        if (p.y_f32)
            ((float *)p.y)[at + j] = e[j];
        else
            ((__bf16 *)p.y)[at + j] = (__bf16)e[j];
    }
}

} /* namespace */

/*
 * FX blocks of 16 tokens and FW of 16 rows of w a workgroup (of two matrices: one
 * block of each, of the same columns).  K blocks go round the NW wavefronts; each
 * has a ring of ST blocks in LDS of its own, filled by direct copies with lanes
 * along rows, so nothing waits at a barrier until the wavefronts join.
 *
 * LDS rows of 128 bytes; a row's 16-byte unit c lies at c ^ (row / 2 % 8), so that
 * the 16 rows of one read take different banks.  A lane of group h reads units 2h
 * and 2h + 1 of both operands: any order of K is right that both share.
 *
 * Memory bounds it for a few tokens: one token by 16384 x 8192, 134 MB, in 31.0 us
 * (4.3 TB/s; a large copy 4.8 to 5.0), by 8192 x 8192 in 14.9, by two of 8192 x 4096
 * in 13.0 with exact sums.  With 64 tokens the copies of x, 16 KB beside 4 of weights
 * a K block and wavefront, count as much: 64 x 8192x8192 in 20.8 us.
 */
template <int FX, int FW, int NW, int ST, bool TWO, bool EXACT>
__global__ __launch_bounds__(NW * 64) void block_rows_kernel(BlockGemmParams p)
{
    static_assert(!TWO || FW == 2, "one block of each of two matrices");
    constexpr int XB = FX * 2048, WB = FW * 2048, SLOT = XB + WB + 256;
    constexpr int LOADS = 2 * FX + 2 * FW + 1;
    constexpr int WAVE = ST * SLOT + FW * 256, OUT = TWO ? 1 : FW;
    static_assert(FX <= 4 && LOADS * (ST - 1) < 64, "ring");
    static_assert(WAVE >= FX * FW * 1024, "the join");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * WAVE];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
    const int32_t n0 = blockIdx.x * (16 * OUT), m0 = blockIdx.y * (16 * FX);
    const uint32_t base = lds_addr(smem) + wave * WAVE;
    uint8_t *mine = smem + wave * WAVE;
    /* this wavefront's blocks: every NW-th of the part's */
    const int32_t part = blockIdx.z, k0 = kslice_begin(p.nk, p.splits, part) + wave, k1 = kslice_begin(p.nk, p.splits, part + 1);
    const int32_t mine_n = k1 > k0 ? (k1 - k0 + NW - 1) / NW : 0;

    /* copy d of 8 rows: lane's row and the unit that belongs at its place */
    const int drow = lane >> 3;
    const i32x4 rx = rsrc_words(p.x + (int64_t)m0 * p.ldx);
    const i32x4 rw = rsrc_words(p.w + (int64_t)n0 * p.ldw), ru = rsrc_words(TWO ? p.up + (int64_t)n0 * p.ldu : p.w);
    uint32_t xoff[2 * FX], woff[2 * FW];
    int32_t unit[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) unit[e] = (lane & 7) ^ ((4 * e + (drow >> 1)) & 7);
#pragma unroll
    for (int d = 0; d < 2 * FX; ++d)
        xoff[d] = m0 + d * 8 + drow < p.M ? (uint32_t)((d * 8 + drow) * (int32_t)p.ldx + unit[d & 1] * 16) : kOOB;
#pragma unroll
    for (int d = 0; d < 2 * FW; ++d) {
        const int r = (TWO ? d & 1 : d) * 8 + drow;
        woff[d] = n0 + r < p.N ? (uint32_t)(r * (int32_t)(TWO && d >= 2 ? p.ldu : p.ldw) + unit[d & 1] * 16) : kOOB;
    }
    /* the scale of the lane's token (rows past the last repeat it) */
    const float *xs = p.xs + std::min(m0 + (lane & (16 * FX - 1)), p.M - 1);

    auto copy = [&](int32_t i, uint32_t slot) __attribute__((always_inline)) {
        const int32_t kb = k0 + i * NW, k = kb * 128;
        const bool in = i < mine_n;
        bool ok[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) ok[e] = in && k + unit[e] * 16 < p.K;
        unroll<2 * FW>([&](auto dc) __attribute__((always_inline)) {
            constexpr int d = decltype(dc)::value;
            dma16<XB + d * 1024>(TWO && d >= 2 ? ru : rw, base + slot, ok[d & 1] && woff[d] != kOOB ? woff[d] + k : kOOB);
        });
        unroll<2 * FX>([&](auto dc) __attribute__((always_inline)) {
            constexpr int d = decltype(dc)::value;
            dma16<d * 1024>(rx, base + slot, ok[d & 1] && xoff[d] != kOOB ? xoff[d] + k : kOOB);
        });
        dma_global4(base + slot + XB + WB, xs + (in ? kb : 0) * p.lxs);
    };
    /* the weights' scales of the next 64 blocks of this wavefront */
    auto copy_scales = [&](int32_t i) __attribute__((always_inline)) {
        const int32_t kb = std::min(k0 + (i + lane) * NW, p.nk - 1);
        unroll<FW>([&](auto fc) __attribute__((always_inline)) {
            constexpr int f = decltype(fc)::value;
            const int32_t n = TWO ? n0 : std::min(n0 + f * 16, p.N - 1);
            const float *s = (TWO && f == 1 ? p.us + (int64_t)(n >> 7) * p.lus : p.ws + (int64_t)(n >> 7) * p.lws) + kb;
            dma_global4(base + ST * SLOT + f * 256, s);
        });
    };

    f32x4 acc[FW][FX];
#pragma unroll
    for (int f = 0; f < FW; ++f)
#pragma unroll
        for (int x = 0; x < FX; ++x) acc[f][x] = f32x4{};

    if (mine_n > 0) {
        copy_scales(0);
        unroll<ST>([&](auto sc) __attribute__((always_inline)) { copy(decltype(sc)::value, decltype(sc)::value * SLOT); });
        const int frow = lane & 15, h = lane >> 4, sw = (frow >> 1) & 7;
        uint32_t slot = 0;
        for (int32_t i = 0; i < mine_n; ++i) {
            if (i && (i & 63) == 0) {
                copy_scales(i);
                wait_vmcnt<0>();
            }
            wait_vmcnt<(ST - 1) * LOADS>();
            if ((p.K & 15) && k0 + i * NW == p.nk - 1) {
                /* K ends inside a unit: what lies behind it becomes zero */
                const int32_t end = p.K - (p.nk - 1) * 128, at = end & ~15;
                for (int r = lane; r < 16 * (FX + FW); r += 64) {
                    const uint32_t row = slot + (r < 16 * FX ? r * 128 : XB + (r - 16 * FX) * 128);
                    uint8_t *u = mine + row + ((at >> 4) ^ ((r >> 1) & 7)) * 16;
                    for (int b = end & 15; b < 16; ++b) u[b] = 0;
                }
            }
            asm volatile("" ::: "memory");
            const uint8_t *s = mine + slot;
            auto frag = [&](int off, int blk) __attribute__((always_inline)) {
                const uint8_t *row = s + off + (blk * 16 + frow) * 128;
                const i32x4 lo = *(const i32x4 *)(row + (((2 * h) ^ sw) << 4));
                const i32x4 hi = *(const i32x4 *)(row + (((2 * h + 1) ^ sw) << 4));
                return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            };
            i32x8 a[FW], b[FX];
            float sw_[FW], sx[FX];
#pragma unroll
            for (int f = 0; f < FW; ++f) {
                a[f] = frag(XB, f);
                sw_[f] = *(const float *)(mine + ST * SLOT + f * 256 + (i & 63) * 4);
            }
#pragma unroll
            for (int x = 0; x < FX; ++x) {
                b[x] = frag(0, x);
                sx[x] = *(const float *)(s + XB + WB + (x * 16 + frow) * 4);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            copy(i + ST, slot);
#pragma unroll
            for (int f = 0; f < FW; ++f)
#pragma unroll
                for (int x = 0; x < FX; ++x) {
                    f32x4 part{};
                    if constexpr (EXACT) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(a[f], j), widen(b[x], j), part, 0, 0, 0);
                    } else {
                        part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[f], b[x], part, 0, 0, 0, 0, 0, 0);
                    }
                    const float sc = sw_[f] * sx[x];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[f][x][e] = __builtin_fmaf(part[e], sc, acc[f][x][e]);
                }
            slot = slot + SLOT == ST * SLOT ? 0 : slot + SLOT;
        }
    }
    /* copies past the last block have landed before their places hold sums */
    wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int f = 0; f < FW; ++f)
#pragma unroll
        for (int x = 0; x < FX; ++x) *(f32x4 *)(mine + (f * FX + x) * 1024 + lane * 16) = acc[f][x];
    __syncthreads();
    /* a lane's four sums: rows 4 (lane / 16) .. of w, token lane % 16 */
    for (int t = threadIdx.x; t < OUT * FX * 64; t += NW * 64) {
        const int l = t & 63, blk = t >> 6, f = blk / FX, x = blk - f * FX;
        const int32_t m = m0 + x * 16 + (l & 15), n = n0 + f * 16 + (l >> 4) * 4;
        f32x4 v{}, u{};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            v += *(const f32x4 *)(smem + w * WAVE + blk * 1024 + l * 16);
            if constexpr (TWO) u += *(const f32x4 *)(smem + w * WAVE + (FX + blk) * 1024 + l * 16);
        }
        if (m >= p.M || n >= p.N) continue;
        const int64_t plane = (int64_t)p.M * p.ldp;
        float *o = p.part + (int64_t)part * p.part_planes * plane + (int64_t)m * p.ldp + n;
        if (TWO && p.part_planes == 2) {
            *(f32x4 *)o = v;
            *(f32x4 *)(o + plane) = u;
            continue;
        }
        if constexpr (TWO) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gated(v[e], u[e], p.act);
        }
        if (p.part_planes)
            *(f32x4 *)o = v;
        else
            store4(p, m, n, v);
    }
}

/* Values of a lane of a 32 x 32 matrix block (token lane % 32; columns 8 q + 4 h .. + 3
 * for q < 4, h = lane / 32) to memory, lanes h = 0 and 1 beside each other. */
struct Place {
    int32_t m, n;                 /* the lane's token, the block's first column */
    int h;
};

/* Swaps the upper 32 lanes of a with the lower 32 of b. */
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

/* Quads FROM .. FROM + QUADS - 1 as the first columns. */
template <int FROM, int QUADS>
__device__ __forceinline__ void store_part(const BlockGemmParams &p, float *plane, const Place &at, const f32x16 &v)
{
#pragma unroll
    for (int q = 0; q < QUADS; ++q) {
        const int32_t n = at.n + 8 * q + 4 * at.h;
        f32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = v[4 * (FROM + q) + e];
        if (at.m < p.M && n < p.N) *(f32x4 *)(plane + (int64_t)at.m * p.ldp + n) = t;
    }
}

template <int QUADS>
__device__ __forceinline__ void store_rows(const BlockGemmParams &p, const Place &at, const f32x16 &v)
{
    if (!p.y_f32) {
        /* 8 columns a lane: quads 0 and 1 (2 and 3) of both halves trade places */
#pragma unroll
        for (int q = 0; q < QUADS; q += 2) {
            uint32_t d[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float a = v[4 * (q + j) + 2 * i], b = v[4 * (q + j) + 2 * i + 1];
                    d[j][i] = pack_bf16(a, b);
                }
            swap32(d[0][0], d[1][0]);
            swap32(d[0][1], d[1][1]);
            const int32_t n = at.n + 8 * (q + at.h);
            if (at.m >= p.M || n >= p.N) continue;
            uint16_t *o = (uint16_t *)p.y + (int64_t)at.m * p.ldy + n;
            if (n + 8 <= p.N) {
                *(u32x4_any *)o = u32x4_any{d[0][0], d[0][1], d[1][0], d[1][1]};
                continue;
            }
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (n + j < p.N) o[j] = (uint16_t)(d[j >> 2][(j >> 1) & 1] >> (16 * (j & 1)));
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < QUADS; ++q) {
        f32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = v[4 * q + e];
        if (at.m < p.M) store4(p, at.m, at.n + 8 * q + 4 * at.h, t);
    }
}

__device__ __forceinline__ void store_codes(const BlockGemmParams &p, const Place &at, const f32x16 &v, float inverse)
{
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = v[4 * q + e] * inverse;
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        d[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
    }
    /* 16 columns a lane: dwords of quads 0, 1 for h = 0, of 2, 3 for h = 1 */
    swap32(d[0], d[2]);
    swap32(d[1], d[3]);
    const int32_t n = at.n + 16 * at.h;
    if (at.m >= p.M || n >= p.N) return;
    uint8_t *o = p.q.codes + (int64_t)at.m * p.q.ld + n;
    if (n + 16 <= p.N) {
        *(uint4 *)o = make_uint4(d[0], d[2], d[1], d[3]);
        return;
    }
    const uint32_t w[4] = {d[0], d[2], d[1], d[3]};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (n + j < p.N) o[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

/*
 * TX tokens and TW rows of w (of two matrices: TW / 2 of each, of the same columns)
 * a tile, a workgroup of WX x WW wavefronts, one K block of 128 a stage of a ring of
 * ST.  A wavefront's block is two by FW matrix blocks of 32 x 32, in a row of two
 * at a time: the sums of a K block come from two instructions each, begun at zero,
 * and the multiply-adds of them into the fp32 sums run while the matrix unit has the
 * instruction behind: the first's during the second's, the second's during the next
 * row's first.  Fragments are read into their own registers again right after their
 * last use.  (FW = 1, for few tokens: the fragments of two K blocks are held, and
 * the sums of two, so that neither LDS nor the multiply-adds are waited for.)
 *
 * A stage is rows of 128 bytes (a row's 16-byte unit c lies at c ^ (row / 2 % 8)),
 * the tokens' scales and the weights'.  Before the last row of matrix blocks of a K
 * block is a barrier: by then every fragment of the stage has been read and the
 * next stage has landed, and the weights' copies of the K block ST ahead follow it.
 * The tokens' fragments have been read by all one row earlier (FW > 2: a second
 * barrier, before row 1), and the tokens' copies go there, so that the copies of a
 * K block come in two bursts.
 *
 * A workgroup takes every gridDim.x-th unit (a tile's part of K).  The first copies
 * of its next unit land before it stores the sums of this one, from registers, and
 * nothing waits for the stores before the unit's second K block.
 *
 * 256 x 256 tiles: 4096 x 8192x8192 in 236 us, 2.33 PFLOP/s.  A K block takes 1.53 us
 * (2.8 PFLOP/s), of which multiply-adds cost a tenth and copies a seventh (with each
 * left out, 8192^3 in 425 and 415 us against 486); matrix instructions run in 0.61 of
 * all cycles at the 1.78 GHz that the power limit leaves.  A tile's begin and stores
 * take some 8 us more.  Copies of a K block in one burst 479 us (8192^3), in two 459;
 * the next unit's copies behind the stores 142 us (8192 x 8192x2048), before them 131.
 * Exact sums (128 x 256): two of 8192 x 4096 by 2048 tokens in 238 us, 1.15 PFLOP/s,
 * where the widening of codes, half as many instruction cycles as the products',
 * stands beside them.
 */
template <int TX, int TW, int WX, int WW, int ST, int MINB, bool TWO, bool EXACT>
__global__ __launch_bounds__(WX *WW * 64, MINB) void block_tile_kernel(BlockGemmParams p)
{
    constexpr int NW = WX * WW, WTX = TX / WX, WTW = TW / WW, FW = WTW / 32;
    constexpr int XB = TX * 128, WB = TW * 128, SCX = XB + WB, SCW = SCX + TX * 4, STAGE = SCW + 256;
    constexpr int SCG = TX / 64 + 1, SL = (SCG + NW - 1) / NW;       /* scale copies of a stage, of a wavefront */
    constexpr int XL = TX / 8 / NW, WL = TW / 8 / NW, LOADS = XL + WL + SL;
    constexpr int OC = TWO ? WTW / 2 : WTW, TN = TWO ? TW / 2 : TW;  /* columns out */
    constexpr int OF = OC < 32 ? 1 : OC / 32, QUADS = OC < 32 ? 2 : 4;
    constexpr bool EARLY = FW > 2;                 /* tokens' copies in row 1 */
    constexpr bool HALVES = TWO && FW == 1;        /* both matrices in one matrix block */
    constexpr bool BY_WAVE = TWO && NW * 8 % WTW == 0;      /* a wavefront copies one of them */
    static_assert(WTX == 64 && NW % 2 == 0 && WTW <= 128 && (ST - 1) * LOADS < 64 && (!EARLY || ST == 2), "tile");
    static_assert(!TWO || OC % (NW * 8) == 0 || BY_WAVE, "a copy is of one matrix");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[ST * STAGE + (TWO && TN == 128 ? WW * TX * 4 : 0)];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wx = wave / WW, ww = wave % WW;
    const int32_t tm = (p.M + TX - 1) / TX, tn = (p.N + TN - 1) / TN, units = tm * tn * p.splits;
    const uint32_t base = lds_addr(smem);
    /* the scale copies of a stage go round the wavefronts (those past the last
     * repeat the first: the same values to the same place) */
    int sg[SL];
    int64_t sc_step[SL];
#pragma unroll
    for (int i = 0; i < SL; ++i) {
        sg[i] = (wave + i * NW) % SCG;
        sc_step[i] = sg[i] < SCG - 1 ? p.lxs : 1;
    }

    /* the unit in hand, and what its copies need of a lane */
    int32_t m0, n0, part, k0, k1, have;
    i32x4 rx, rw, ru;
    uint32_t xoff[XL], woff[WL];
    const float *sc[SL];
    int lane, unit;
    auto setup = [&](int32_t id) __attribute__((always_inline)) {
        /* formed from a lane index that the compiler cannot see through, or it
         * would hold all of this across units */
        lane = lane_id();
        asm volatile("" : "+v"(lane));
        part = id / (tm * tn);
        const int32_t t = id - part * (tm * tn);
        /* neighbouring units share operands: bands of 4 rows of tiles */
        const int32_t band = t / (4 * tn), in = t - band * 4 * tn, high = std::min(4, tm - band * 4);
        m0 = (band * 4 + in % high) * TX;
        n0 = in / high * TN;
        k0 = kslice_begin(p.nk, p.splits, part);
        k1 = kslice_begin(p.nk, p.splits, part + 1);
        /* copy d of 8 rows: the lane's row, and the unit that belongs at its place
         * (rows of d and d + 1 are NW * 8 apart: a multiple of 16) */
        const int drow = lane >> 3;
        unit = (lane & 7) ^ ((4 * wave + (drow >> 1)) & 7);
        rx = rsrc_words(p.x + (int64_t)m0 * p.ldx);
        rw = rsrc_words(p.w + (int64_t)n0 * p.ldw);
        if constexpr (TWO) ru = rsrc_words(p.up + (int64_t)n0 * p.ldu);
        const bool second = BY_WAVE && wave * 8 % WTW >= OC;       /* this wavefront copies up */
        if (second) rw = ru;
#pragma unroll
        for (int d = 0; d < XL; ++d) {
            const int r = (d * NW + wave) * 8 + drow;
            xoff[d] = m0 + r < p.M ? (uint32_t)(r * (int32_t)p.ldx + unit * 16) : kOOB;
        }
#pragma unroll
        for (int d = 0; d < WL; ++d) {
            int r = (d * NW + wave) * 8 + drow;
            if constexpr (TWO) r = r / WTW * OC + r % OC;
            const bool u = BY_WAVE ? second : TWO && (d * NW * 8 / OC) % 2 == 1;
            woff[d] = n0 + r < p.N ? (uint32_t)(r * (int32_t)(u ? p.ldu : p.ldw) + unit * 16) : kOOB;
        }
        /* rows past the last repeat its scale */
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            if (sg[i] < SCG - 1)
                sc[i] = p.xs + std::min(m0 + sg[i] * 64 + lane, p.M - 1);
            else if (TWO)
                sc[i] = lane & 1 ? p.us + (int64_t)(n0 >> 7) * p.lus : p.ws + (int64_t)(n0 >> 7) * p.lws;
            else
                sc[i] = p.ws + (int64_t)(std::min(n0 + (lane & 1) * 128, p.N - 1) >> 7) * p.lws;
            sc[i] += k0 * sc_step[i];
        }
        /* K blocks whose unit of this lane lies before K, in this part */
        have = std::min(k1, (p.K - unit * 16 + 127) >> 7);
    };
    auto copy = [&](auto dc, int32_t kb, uint32_t so) __attribute__((always_inline)) {
        constexpr int d = decltype(dc)::value;
        /* kOOB and an offset along a row stay out of range */
        const uint32_t k = (uint32_t)kb * 128;
        if constexpr (d < XL) {
            dma16<d * NW * 1024>(rx, base + so + wave * 1024, kb < have ? xoff[d] + k : kOOB);
        } else if constexpr (d < XL + WL) {
            dma16<XB + (d - XL) * NW * 1024>(TWO && !BY_WAVE && ((d - XL) * NW * 8 / OC) % 2 == 1 ? ru : rw, base + so + wave * 1024,
                                             kb < have ? woff[d - XL] + k : kOOB);
        } else {
            constexpr int i = d - XL - WL;
            dma_global4(base + so + SCX + sg[i] * 256, sc[i]);
            if (kb + 1 < k1) sc[i] += sc_step[i];
        }
    };
    auto first_copies = [&]() __attribute__((always_inline)) {
        if (k1 <= k0) return;
        unroll<ST>([&](auto tc) __attribute__((always_inline)) {
            constexpr int t = decltype(tc)::value;
            unroll<LOADS>([&](auto dc) __attribute__((always_inline)) { copy(dc, k0 + t, (uint32_t)(t * STAGE)); });
        });
    };
    /* K ends inside a unit: the lanes that copied it clear what lies behind, once it
     * has landed */
    auto clear_tail = [&](int32_t kb, uint32_t so) __attribute__((always_inline)) {
        if ((p.K & 15) == 0 || kb != p.nk - 1 || kb >= k1) return;
        const int32_t left = p.K - kb * 128 - unit * 16;
        if (left > 0 && left < 16) {
            const uint64_t lo = left >= 8 ? ~0ull : (1ull << (8 * left)) - 1, hi = left <= 8 ? 0 : (1ull << (8 * (left - 8))) - 1;
            uint64_t *u = (uint64_t *)(smem + so + wave * 1024 + lane * 16);
#pragma unroll 1
            for (int d = 0; d < XL + WL; ++d, u += NW * 128) {
                u[0] &= lo;
                u[1] &= hi;
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };

    const int32_t round = xcd_remap(blockIdx.x, gridDim.x);
    int32_t id = round;
    if (id >= units) return;
    setup(id);
    first_copies();
    if (k1 > k0) wait_vmcnt<(ST - 1) * LOADS>();
    int ahead = 0;                /* K blocks that need no wait: they have landed */
    for (;;) {
        f32x16 acc[FW][2];
#pragma unroll
        for (int f = 0; f < FW; ++f)
#pragma unroll
            for (int x = 0; x < 2; ++x) acc[f][x] = f32x16{};

        if (k1 > k0) {
            const int frow = lane & 31, h = lane >> 5, sw = (frow >> 1) & 7;
            auto frag = [&](uint32_t rows, int s) __attribute__((always_inline)) {
                const uint8_t *row = smem + rows + frow * 128;
                const i32x4 lo = *(const i32x4 *)(row + (((4 * s + 2 * h) ^ sw) << 4));
                const i32x4 hi = *(const i32x4 *)(row + (((4 * s + 2 * h + 1) ^ sw) << 4));
                return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            };
            if constexpr (FW == 1) {
                /* both K blocks' fragments in registers: a K block's are read while the
                 * one before it is multiplied */
                i32x8 xf[2][2][2], wf[2][2];
                float sx[2][2], sw_[2][2], by[2][2];
                f32x16 sum[2][2];
                auto read = [&](auto bc, uint32_t so, int part) __attribute__((always_inline)) {
                    constexpr int b = decltype(bc)::value;
                    if (part < 2) {
                        wf[b][part] = frag(so + XB + ww * WTW * 128, part);
                        xf[b][0][part] = frag(so + wx * WTX * 128, part);
                        return;
                    }
                    xf[b][1][part - 2] = frag(so + (wx * WTX + 32) * 128, part - 2);
                    if (part == 3) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) sx[b][x] = *(const float *)(smem + so + SCX + (wx * WTX + x * 32 + frow) * 4);
                        sw_[b][0] = *(const float *)(smem + so + SCW + (TWO ? 0 : ww * WTW / 128 * 4));
                        sw_[b][1] = TWO ? *(const float *)(smem + so + SCW + 4) : 0.0f;
                    }
                };
                auto multiply = [&](auto bc, int x, int s) __attribute__((always_inline)) {
                    constexpr int b = decltype(bc)::value;
                    f32x16 v = s ? sum[b][x] : f32x16{};
                    if constexpr (EXACT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(wf[b][s], i), widen(xf[b][x][s], i), v, 0, 0, 0);
                    } else {
                        v = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[b][s], xf[b][x][s], v, 0, 0, 0, 0, 0, 0);
                    }
                    sum[b][x] = v;
                };
                auto add = [&](auto bc, int x) __attribute__((always_inline)) {
                    constexpr int b = decltype(bc)::value;
                    const float s0 = by[0][x], s1 = by[1][x];
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[0][x][e] = __builtin_fmaf(sum[b][x][e], HALVES && e >= 8 ? s1 : s0, acc[0][x][e]);
                    asm volatile("" : "+v"(acc[0][x]));
                };
                auto fence = []() __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
                typedef std::integral_constant<int, 0> Zero;
                typedef std::integral_constant<int, 1> One;
                clear_tail(k0, 0);
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) read(Zero{}, 0, i);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    sum[1][x] = f32x16{};
                    by[0][x] = by[1][x] = 0.0f;
                }
                uint32_t so = 0;
                auto block = [&](auto bc, int32_t kb) __attribute__((always_inline)) {
                    constexpr int b = decltype(bc)::value;
                    typedef std::integral_constant<int, 1 - b> Other;
                    const uint32_t next = so + STAGE == ST * STAGE ? 0 : so + STAGE;
                    auto copies = [&](auto qc) __attribute__((always_inline)) {
                        constexpr int q = decltype(qc)::value;
                        unroll<LOADS>([&](auto dc) __attribute__((always_inline)) {
                            if constexpr (decltype(dc)::value * 4 / LOADS == q) copy(dc, kb + ST, so);
                        });
                    };
                    /* this K block's fragments are here, from every wavefront's view:
                     * its stage is free, and the next has landed */
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (ahead > 0)
                        --ahead;
                    else
                        wait_vmcnt<(ST - 2) * LOADS>();
                    clear_tail(kb + 1, next);
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    unroll<4>([&](auto ic) __attribute__((always_inline)) {
                        constexpr int i = decltype(ic)::value;
                        multiply(bc, i & 1, i >> 1);
                        fence();
                        read(Other{}, next, i);
                        copies(ic);
                        if constexpr (i >= 2) add(Other{}, i - 2);
                        fence();
                    });
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        by[0][x] = sx[b][x] * sw_[b][0];
                        by[1][x] = sx[b][x] * sw_[b][1];
                    }
                    so = next;
                };
                int32_t kb = k0;
                for (; kb + 1 < k1; kb += 2) {
                    block(Zero{}, kb);
                    block(One{}, kb + 1);
                }
                if (kb < k1) {
                    block(Zero{}, kb);
                    add(Zero{}, 0);
                    add(Zero{}, 1);
                } else {
                    add(One{}, 0);
                    add(One{}, 1);
                }
            } else {
                i32x8 xf[2][2], wf[2];
                float sx[2], sw_[2];
                auto read_w = [&](uint32_t so, int f, int s) __attribute__((always_inline)) {
                    wf[s] = frag(so + XB + (ww * WTW + f * 32) * 128, s);
                };
                auto read_x = [&](uint32_t so, int x, int s) __attribute__((always_inline)) {
                    xf[x][s] = frag(so + (wx * WTX + x * 32) * 128, s);
                };
                auto read_scales = [&](uint32_t so) __attribute__((always_inline)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) sx[x] = *(const float *)(smem + so + SCX + (wx * WTX + x * 32 + frow) * 4);
                    sw_[0] = *(const float *)(smem + so + SCW + (TWO ? 0 : ww * WTW / 128 * 4));
                    sw_[1] = TWO ? *(const float *)(smem + so + SCW + 4) : 0.0f;
                };

                /* the unit's first K block has landed */
                clear_tail(k0, 0);
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    read_x(0, 0, s);
                    read_x(0, 1, s);
                    read_w(0, 0, s);
                }
                read_scales(0);

                f32x16 sum[2];
                float scale[2][2], last = 0.0f, last2 = 0.0f;
                sum[0] = sum[1] = f32x16{};
                uint32_t so = 0;
                auto multiply = [&](int x, int s) __attribute__((always_inline)) {
                    f32x16 v = s ? sum[x] : f32x16{};
                    if constexpr (EXACT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(wf[s], i), widen(xf[x][s], i), v, 0, 0, 0);
                    } else {
                        v = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[s], xf[x][s], v, 0, 0, 0, 0, 0, 0);
                    }
                    sum[x] = v;
                };
                auto add = [&](f32x16 &a, int x, float by, float by2) __attribute__((always_inline)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) a[e] = __builtin_fmaf(sum[x][e], HALVES && e >= 8 ? by2 : by, a[e]);
                    /* here, not where the sums are next used */
                    asm volatile("" : "+v"(a));
                };
                auto fence = []() __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
                for (int32_t kb = k0; kb < k1; ++kb) {
                    const uint32_t next = so + STAGE == ST * STAGE ? 0 : so + STAGE;
                    unroll<FW>([&](auto fc) __attribute__((always_inline)) {
                        constexpr int f = decltype(fc)::value;
                        constexpr bool end = f == FW - 1;
                        constexpr int m = TWO && !HALVES && f >= FW / 2 ? 1 : 0;
                        /* this row's copies: a quarter behind each instruction */
                        constexpr int c0 = EARLY && end ? XL : 0, c1 = EARLY ? f == 1 ? XL : end ? LOADS : 0 : end ? LOADS : 0;
                        auto copies = [&](auto qc) __attribute__((always_inline)) {
                            constexpr int q = decltype(qc)::value;
                            unroll<LOADS>([&](auto dc) __attribute__((always_inline)) {
                                constexpr int d = decltype(dc)::value;
                                if constexpr (d >= c0 && d < c1 && (d - c0) * 4 / (c1 - c0) == q) copy(dc, kb + ST, so);
                            });
                        };
                        if constexpr (EARLY && f == 1) {
                            __builtin_amdgcn_s_barrier();
                            asm volatile("" ::: "memory");
                        }
                        if constexpr (end) {
                            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                            /* (of a workgroup's later units the first ST have landed
                             * before: stores of the unit before are not waited for yet) */
                            if (ahead > 0)
                                --ahead;
                            else
                                wait_vmcnt<(ST - 2) * LOADS + (EARLY ? XL : 0)>();
                            clear_tail(kb + 1, next);
                            __builtin_amdgcn_s_barrier();
                            asm volatile("" ::: "memory");
                        }
                        multiply(0, 0);
                        fence();
                        if constexpr (end) read_x(next, 0, 0);
                        copies(std::integral_constant<int, 0>{});
                        /* the row before: of the K block before for the first */
                        add(acc[f == 0 ? FW - 1 : f - 1][1], 1, f == 0 ? last : scale[TWO && f - 1 >= FW / 2 ? 1 : 0][1], last2);
                        fence();
                        multiply(1, 0);
                        fence();
                        if constexpr (f == 0) {
                            /* not before: their reads were the last ones */
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                scale[0][x] = sx[x] * sw_[0];
                                if (TWO) scale[1][x] = sx[x] * sw_[1];
                            }
                        }
                        read_w(end ? next : so, end ? 0 : f + 1, 0);
                        if constexpr (end) read_x(next, 1, 0);
                        copies(std::integral_constant<int, 1>{});
                        fence();
                        multiply(0, 1);
                        fence();
                        if constexpr (end) read_x(next, 0, 1);
                        copies(std::integral_constant<int, 2>{});
                        fence();
                        multiply(1, 1);
                        fence();
                        read_w(end ? next : so, end ? 0 : f + 1, 1);
                        if constexpr (end) {
                            read_x(next, 1, 1);
                            read_scales(next);
                        }
                        copies(std::integral_constant<int, 3>{});
                        add(acc[f][0], 0, scale[m][0], scale[TWO ? 1 : 0][0]);
                        fence();
                    });
                    last = scale[TWO && !HALVES ? 1 : 0][1];
                    if (HALVES) last2 = scale[1][1];
                    so = next;
                }
                add(acc[FW - 1][1], 1, last, last2);
            }
        }

        /* every fragment has been read and the copies of K blocks past the last have
         * landed: the ring is free for the next unit */
        wait_vmcnt<0>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int32_t mw = m0 + wx * WTX, nw = n0 + ww * OC, nb = n0 >> 7, from = part;
        id += gridDim.x;
        const bool more = id < units;
        if (more) {
            setup(id);
            first_copies();
        }

        int el = lane_id();
        asm volatile("" : "+v"(el));
        const int h = el >> 5;
        const bool activate = TWO && (p.part_planes < 2);
        if constexpr (TWO) {
            if (activate) {
#pragma unroll
                for (int f = 0; f < OF; ++f)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int e = 0; e < 4 * QUADS; ++e) {
                            const float a = acc[f][x][e], b = HALVES ? acc[f][x][8 + e] : acc[(OF + f) % FW][x][e];
                            acc[f][x][e] = gated(a, b, p.act);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
        }
        if (more) {
            wait_vmcnt<0>();
            ahead = ST - 1;
        }
        if (p.part_planes) {
            const int64_t plane = (int64_t)p.M * p.ldp;
            float *o = p.part + (int64_t)from * p.part_planes * plane;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int f = 0; f < OF; ++f) {
                    const Place at{mw + x * 32 + (el & 31), nw + f * 32, h};
                    store_part<0, QUADS>(p, o, at, acc[f][x]);
                    if constexpr (TWO)
                        if (!activate) store_part<HALVES ? 2 : 0, QUADS>(p, o + plane, at, acc[(OF + f) % FW][x]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        } else if (TWO && TN == 128 && p.q.codes) {
            if constexpr (TWO && TN == 128) {
            /* a row's 128 columns are those of the WW wavefronts beside each other */
            float *red = (float *)(smem + ST * STAGE);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float a = 0.0f;
#pragma unroll
                for (int f = 0; f < OF; ++f)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float v = acc[f][x][e];
                        a = fmaxf(a, fabsf(v));
                    }
                a = fmaxf(a, __shfl_xor(a, 32, 64));
                red[ww * TX + wx * WTX + x * 32 + (el & 31)] = a;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float a = 0.0f;
#pragma unroll
                for (int w = 0; w < WW; ++w) a = fmaxf(a, red[w * TX + wx * WTX + x * 32 + (el & 31)]);
                const bool none = a < 0x1p-100f;
                const float inverse = none ? 1.0f : 448.0f / a;
                const int32_t m = mw + x * 32 + (el & 31);
                if (ww == 0 && h == 0 && m < p.M) p.q.scales[(int64_t)nb * p.q.lds + m] = none ? 1.0f : a / 448.0f;
#pragma unroll
                for (int f = 0; f < OF; ++f) {
                    store_codes(p, Place{m, nw + f * 32, h}, acc[f][x], inverse);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            }
        } else {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int f = 0; f < OF; ++f) {
                    store_rows<QUADS>(p, Place{mw + x * 32 + (el & 31), nw + f * 32, h}, acc[f][x]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        if (!more) break;
    }
}

/*
 * Some tokens, a stream of weights: 128 tokens and 32 rows of w (of two matrices 16 of
 * each) a workgroup.  Memory answers after some 2 us, the caches, where x comes from,
 * after less than one, and a wavefront's copies land in order: so they are made by
 * wavefronts of their own, two that keep a ring of XS steps of x filled and one for a
 * ring of WS of w.  Four multiply, 32 tokens each.  A step is B K blocks, whose
 * fragments are read while the step before is multiplied; all meet at one barrier a
 * step.
 *
 * 128 x 8192x8192: 23.6 us, where the tiles of 128 x 64 take 31.8 and, in two parts,
 * 25.8; 128 x 4096x4096 11.0 against 15.6.  Without any data (every copy out of
 * range) it takes 17.8 of 26.6 us with a step of one K block: the chain of barrier,
 * fragments and products; x, 16 KB a K block from the L2, and the weights' 4 KB from
 * memory add to it.  A second wavefront for the weights, or four for x, changed
 * nothing.
 */
template <int B, int XS, int WS, bool TWO, bool EXACT>
__global__ __launch_bounds__(448) void block_stream_kernel(BlockGemmParams p)
{
    constexpr int TX = 128;
    constexpr int XBLOCK = TX * 128 + TX * 4, WBLOCK = 4096 + 256, W0 = XS * B * XBLOCK;
    constexpr int XL = TX / 16;                             /* copies of a block's rows */
    static_assert(XS >= 2 && WS >= 2 && (XS - 1) * B * (XL + 1) < 64 && (WS - 1) * B * 5 < 64, "rings");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[W0 + WS * B * WBLOCK];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
    constexpr int COLS = TWO ? 16 : 32;
    const int32_t n0 = blockIdx.x * COLS, m0 = blockIdx.y * TX, part = blockIdx.z;
    const int32_t k0 = kslice_begin(p.nk, p.splits, part), k1 = kslice_begin(p.nk, p.splits, part + 1);
    const int32_t steps = (k1 - k0 + B - 1) / B;
    const uint32_t base = lds_addr(smem);

    if (wave >= 4) {
        /* copies: 8 rows each, the lane's row and the 16-byte unit that belongs at its
         * place, c ^ (row / 2 % 8) */
        const int drow = lane >> 3, pw = wave - 4;
        int32_t unit[2], have[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            unit[e] = (lane & 7) ^ ((4 * e + (drow >> 1)) & 7);
            have[e] = std::min(k1, (p.K - unit[e] * 16 + 127) >> 7);
        }
        auto stream = [&](auto is_w) __attribute__((always_inline)) {
            constexpr bool W = decltype(is_w)::value;
            constexpr int N = W ? 4 : XL, RING = W ? WS : XS, BLOCK = W ? WBLOCK : XBLOCK, LOADS = B * (N + 1);
            const uint8_t *from = W ? p.w + (int64_t)n0 * p.ldw : p.x + (int64_t)m0 * p.ldx;
            const i32x4 r0 = rsrc_words(from), r1 = rsrc_words(W && TWO ? p.up + (int64_t)n0 * p.ldu : from);
            uint32_t off[N];
#pragma unroll
            for (int d = 0; d < N; ++d) {
                const int r = (W ? (TWO ? d & 1 : d) : pw * N + d) * 8 + drow;
                const bool in = W ? n0 + r < p.N : m0 + r < p.M;
                off[d] = in ? (uint32_t)(r * (int32_t)(W ? (TWO && d >= 2 ? p.ldu : p.ldw) : p.ldx) + unit[d & 1] * 16) : kOOB;
            }
            /* scales: of w the lanes of an odd index take the second matrix's, of x each
             * of the two wavefronts 64 tokens'; rows past the last repeat its, blocks
             * past the last too (their codes are zeros) */
            const float *sc;
            if (W)
                sc = TWO && (lane & 1) ? p.us + (int64_t)(n0 >> 7) * p.lus : p.ws + (int64_t)(n0 >> 7) * p.lws;
            else
                sc = p.xs + std::min(m0 + pw * 64 + lane, p.M - 1);
            const int64_t step = W ? 1 : p.lxs;
            sc += k0 * step;
            const uint32_t ring = W ? W0 : 0, rows = W ? 0 : pw * N * 1024, scales = W ? 4096 : TX * 128 + pw * 256;
            auto copy = [&](int32_t kb, uint32_t so) __attribute__((always_inline)) {
                unroll<B>([&](auto jc) __attribute__((always_inline)) {
                    constexpr int j = decltype(jc)::value;
                    unroll<N>([&](auto dc) __attribute__((always_inline)) {
                        constexpr int d = decltype(dc)::value;
                        dma16<j * BLOCK + d * 1024>(W && TWO && d >= 2 ? r1 : r0, base + ring + so + rows,
                                                    kb + j < have[d & 1] ? off[d] + (uint32_t)(kb + j) * 128 : kOOB);
                    });
                    dma_global4(base + ring + so + j * BLOCK + scales, sc);
                    if (kb + j + 1 < k1) sc += step;
                });
            };
            /* K ends inside a unit: the lanes that copied it clear what lies behind */
            auto clear_tail = [&](int32_t kb, uint32_t so) __attribute__((always_inline)) {
                const int32_t end = p.nk - 1;
                if ((p.K & 15) == 0 || kb > end || kb + B <= end || end >= k1) return;
                for (int d = 0; d < N; ++d) {
                    const int32_t left = p.K - end * 128 - unit[d & 1] * 16;
                    uint8_t *u = smem + ring + so + (end - kb) * BLOCK + rows + d * 1024 + lane * 16;
                    for (int b = left; left > 0 && b < 16; ++b) u[b] = 0;
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            };
            unroll<RING>([&](auto tc) __attribute__((always_inline)) {
                constexpr int t = decltype(tc)::value;
                copy(k0 + t * B, (uint32_t)(t * B * BLOCK));
            });
            wait_vmcnt<(RING - 1) * LOADS>();
            clear_tail(k0, 0);
            __builtin_amdgcn_s_barrier();
            uint32_t so = 0;
            for (int32_t i = 0, kb = k0; i < steps; ++i, kb += B) {
                const uint32_t next = so + B * BLOCK == RING * B * BLOCK ? 0 : so + B * BLOCK;
                wait_vmcnt<(RING - 2) * LOADS>();
                clear_tail(kb + B, next);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                copy(kb + RING * B, so);
                so = next;
            }
            wait_vmcnt<0>();
        };
        if (steps > 0) {
            if (pw == 2)
                stream(std::true_type{});
            else
                stream(std::false_type{});
        }
        return;
    }

    const int wt = wave;                                    /* tokens 32 wt .. */
    constexpr int S = 2;                                    /* instructions a K block */
    f32x16 acc{};
    if (steps > 0) {
        const int frow = lane & 31, h = lane >> 5, sw = (frow >> 1) & 7;
        i32x8 xf[2][B][S], wf[2][B][S];
        float sx[2][B], s0[2][B], s1[2][B], by0[B], by1[B];
        f32x16 sum[2][B];
        auto frag = [&](uint32_t rows, int s) __attribute__((always_inline)) {
            const uint8_t *row = smem + rows + frow * 128;
            const int c = 4 * s + 2 * h;
            const i32x4 lo = *(const i32x4 *)(row + ((c ^ sw) << 4));
            const i32x4 hi = *(const i32x4 *)(row + (((c + 1) ^ sw) << 4));
            return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        auto read = [&](int b, uint32_t xo, uint32_t wo) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const uint32_t xj = xo + j * XBLOCK, wj = W0 + wo + j * WBLOCK;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    wf[b][j][s] = frag(wj, s);
                    xf[b][j][s] = frag(xj + wt * 4096, s);
                }
                sx[b][j] = *(const float *)(smem + xj + TX * 128 + (wt * 32 + frow) * 4);
                s0[b][j] = *(const float *)(smem + wj + 4096);
                if (TWO) s1[b][j] = *(const float *)(smem + wj + 4096 + 4);
            }
        };
        auto add = [&](int b, int j) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = __builtin_fmaf(sum[b][j][e], TWO && e >= 8 ? by1[j] : by0[j], acc[e]);
            asm volatile("" : "+v"(acc));
        };
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(0, 0, 0);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            sum[1][j] = f32x16{};
            by0[j] = by1[j] = 0.0f;
        }
        uint32_t xo = 0, wo = 0;
        auto block = [&](auto bc) __attribute__((always_inline)) {
            constexpr int b = decltype(bc)::value;
            xo = xo + B * XBLOCK == XS * B * XBLOCK ? 0 : xo + B * XBLOCK;
            wo = wo + B * WBLOCK == WS * B * WBLOCK ? 0 : wo + B * WBLOCK;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            read(1 - b, xo, wo);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                f32x16 v{};
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if constexpr (EXACT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(wf[b][j][s], i), widen(xf[b][j][s], i), v, 0, 0, 0);
                    } else {
                        v = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[b][j][s], xf[b][j][s], v, 0, 0, 0, 0, 0, 0);
                    }
                }
                sum[b][j] = v;
                add(1 - b, j);
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                by0[j] = sx[b][j] * s0[b][j];
                if (TWO) by1[j] = sx[b][j] * s1[b][j];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        int32_t i = 0;
        for (; i + 1 < steps; i += 2) {
            block(std::integral_constant<int, 0>{});
            block(std::integral_constant<int, 1>{});
        }
        if (i < steps) {
            block(std::integral_constant<int, 0>{});
#pragma unroll
            for (int j = 0; j < B; ++j) add(0, j);
        } else {
#pragma unroll
            for (int j = 0; j < B; ++j) add(1, j);
        }
    }
    const Place at{m0 + wt * 32 + (lane & 31), n0, lane >> 5};
    const int64_t plane = (int64_t)p.M * p.ldp;
    float *o = p.part + (int64_t)part * p.part_planes * plane;
    constexpr int QUADS = TWO ? 2 : 4;
    if (TWO && p.part_planes == 2) {
        store_part<0, QUADS>(p, o, at, acc);
        store_part<TWO ? 2 : 0, QUADS>(p, o + plane, at, acc);
        return;
    }
    if constexpr (TWO) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = acc[e], b = acc[8 + e];
            acc[e] = gated(a, b, p.act);
        }
    }
    if (p.part_planes)
        store_part<0, QUADS>(p, o, at, acc);
    else
        store_rows<QUADS>(p, at, acc);
}

/* One row's 128 columns to 16 lanes: the sum over the parts in ascending order (of
 * both planes where there are two), the activation, and rows or codes.  A second
 * kernel costs some 5 us between calls (3.8 of its own where it has little to do), so
 * parts pay only where tiles are few. */
__global__ __launch_bounds__(256) void block_finish_kernel(BlockGemmParams p)
{
    const int32_t nb = (p.N + 127) >> 7, mb = blockIdx.x / nb, kb = blockIdx.x - mb * nb;
    const int32_t m = mb * 16 + (threadIdx.x >> 4), n = kb * 128 + (threadIdx.x & 15) * 8;
    const int64_t plane = (int64_t)p.M * p.ldp;
    f32x4 v[2] = {}, u[2] = {};
    const bool in = m < p.M && n < p.N;
    if (in) {
        const float *o = p.part + (int64_t)m * p.ldp + n;
        for (int32_t s = 0; s < p.splits; ++s, o += p.part_planes * plane)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                /* ldp is a multiple of 4, and at least N */
                if (n + 4 * j >= p.N) continue;
                const f32x4 a = *(const f32x4 *)(o + 4 * j);
                v[j] = s ? v[j] + a : a;       /* a zero keeps its sign */
                if (p.part_planes < 2) continue;
                const f32x4 b = *(const f32x4 *)(o + plane + 4 * j);
                u[j] = s ? u[j] + b : b;
            }
    }
    float e[8], a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float g = v[j >> 2][j & 3], t = u[j >> 2][j & 3];
        e[j] = p.part_planes == 2 ? gated(g, t, p.act) : g;
        if (n + j >= p.N) e[j] = 0.0f;
        a = fmaxf(a, fabsf(e[j]));
    }
    if (!p.q.codes) {
        if (!in) return;
        store4(p, m, n, f32x4{e[0], e[1], e[2], e[3]});
        if (n + 4 < p.N) store4(p, m, n + 4, f32x4{e[4], e[5], e[6], e[7]});
        return;
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) a = fmaxf(a, __shfl_xor(a, o, 64));
    if (!in) return;
    const bool none = a < 0x1p-100f;
    const float inverse = none ? 1.0f : 448.0f / a;
    if ((threadIdx.x & 15) == 0) p.q.scales[(int64_t)kb * p.q.lds + m] = none ? 1.0f : a / 448.0f;
    uint8_t *c = p.q.codes + (int64_t)m * p.q.ld + n;
    int w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        w[j] = __builtin_amdgcn_cvt_pk_fp8_f32(e[4 * j] * inverse, e[4 * j + 1] * inverse, 0, false);
        w[j] = __builtin_amdgcn_cvt_pk_fp8_f32(e[4 * j + 2] * inverse, e[4 * j + 3] * inverse, w[j], true);
    }
    if (n + 8 <= p.N) {
        *(uint2 *)c = make_uint2((uint32_t)w[0], (uint32_t)w[1]);
        return;
    }
    for (int j = 0; n + j < p.N; ++j) c[j] = (uint8_t)((uint32_t)w[j >> 2] >> (8 * (j & 3)));
}

namespace {

/* Forms of the kernels: tokens and rows of w a workgroup, workgroups that run at once
 * on a compute unit; and the time of one, in us: `begin` and, for each K block, `full`
 * where the device is full of them and `least` where it is not (with `exact` times
 * that for exact sums).  Fitted to timed calls of every form with 1 to 16 parts of K
 * over 162 sizes (one to 4096 tokens, 128 to 16384 columns, K of 500 to 8192; a
 * matrix or two; bf16, codes, fp32): the form that the times choose takes 1.016 of
 * the best form's time in geometric mean.  us of one form and of the next best:
 *   1 x 8192x8192       rows of 16 with 8 wavefronts 16.1, with 4 (two workgroups a
 *                       unit) 16.9;  1 x 16384x8192  28.7, 28.6;  1 x 12000x2048
 *                       9.7, 7.8
 *   24 x 8192x8192      rows of 32 17.3, of 64 18.8;  48 x 8192x8192  28.7, 20.2
 *   64 x 12000x2048     rows of 64 12.6, two workgroups a unit 9.6;  64 x 2048x8192
 *                       11.7, 18.4;  rows of 32 with 8 wavefronts and one
 *                       workgroup a unit are no faster than with 4 and two (24 x
 *                       8192x8192 17.4, 17.5;  24 x 10000x4096  16.8, 15.1)
 *   200 x 4096x4096     stream 12.1, rows of 64 16.3, tiles 128 x 64 16.5
 *   128 x 16384x8192    tiles 128 x 64 38.7, stream 49.9;  100 x 8192x8192  in two
 *                       parts 24.6, 24.2
 *   512 x 8192x8192     tiles 128 x 128 45.9, 128 x 64 59.1, of two workgroups a unit
 *                       59.3 (two parts 54.5)
 *   2048 x 4096x4096    two workgroups a unit 41.9, one 46.4, tiles 256 x 256 48.5
 *   4096 x 4096x4096    tiles 256 x 256 66.9, 128 x 256 75.9;  1024 x 8192x8192  87.4,
 *                       73.4;  into codes, two of 4096x4096  tiles 128 x 256 240, 128 x
 *                       128 269 */
enum { ROWS16, ROWS16_PAIR, ROWS32, ROWS64, ROWS64_PAIR, STREAM, TILE_64, TILE_128, TILE_128_PAIR, TILE_256, TILE_WIDE, FORMS };
struct Form {
    int32_t tx, tw, resident;
    double begin, least, full, exact;
};
constexpr Form kForms[FORMS] = {
    {16, 32, 1, 1.5, 0.068, 0.13, 1.0},  {16, 32, 2, 0.62, 0.094, 0.29, 1.0}, {32, 32, 2, 1.3, 0.093, 0.30, 1.0},
    {64, 32, 1, 2.5, 0.14, 0.19, 1.1},   {64, 32, 2, 2.4, 0.23, 0.28, 1.4},    {128, 32, 1, 2.0, 0.21, 0.25, 1.4},
    {128, 64, 1, 3.1, 0.34, 0.34, 1.8},  {128, 128, 1, 3.8, 0.44, 0.54, 1.9},  {128, 128, 2, 4.0, 0.65, 1.1, 1.6},
    {256, 256, 1, 6.6, 1.2, 1.6, 0.0},   {128, 256, 1, 5.3, 0.80, 0.95, 1.7}};

/* fp32 planes of [M][ldp] that a part of K leaves: a scale of codes needs 128 columns
 * in one workgroup. */
int32_t planes_of(const BlockGemmParams &p, int32_t form, int32_t splits)
{
    return splits > 1 ? 1 + p.two : p.q.codes && form < TILE_256 ? 1 : 0;
}

int64_t units_of(const BlockGemmParams &p, int32_t form)
{
    const int64_t tx = kForms[form].tx, tn = kForms[form].tw >> p.two;
    return (p.M + tx - 1) / tx * ((p.N + tn - 1) / tn);
}

double time_of(const BlockGemmParams &p, int32_t form, int32_t splits, int32_t cus)
{
    const Form &f = kForms[form];
    const int64_t units = units_of(p, form) * splits, most = (int64_t)f.resident * cus, rounds = (units + most - 1) / most;
    const double load = (double)units / (double)(rounds * most);
    const double block = std::max(f.least, f.full * load) * (p.exact ? f.exact : 1.0);
    const double tiles = 2.0 + (double)rounds * (f.begin + (double)((p.nk + splits - 1) / splits) * block);
    /* weights at 5.2 TB/s, x at 20 */
    const double memory = 2.5 + (1.0 + p.two) * (double)p.N * (double)p.K / 5.2e6 + (double)p.M * (double)p.K / 2e7;
    const int32_t planes = planes_of(p, form, splits);
    /* the second kernel, and its planes there and back */
    const double finish = planes ? 5.0 + 1.4e-6 * planes * splits * (double)p.M * (double)p.N : 0.0;
    /* the shorter of the two is not all hidden */
    return std::max(tiles, memory) + 0.1 * std::min(tiles, memory) + finish;
}

} /* namespace */

int64_t block_plan(BlockGemmParams &p, int32_t splits, int32_t cus)
{
    p.exact = p.q.codes || p.y_f32;
    p.form = TILE_128;
    p.splits = 1;
    double best = 1e300;
    for (int32_t form = 0; form < FORMS; ++form) {
        const int32_t tx = kForms[form].tx;
        if (form == TILE_256 && p.exact) continue;      /* its registers are full */
        /* rows and streams are for weights that pass by few tokens (4096 x 256x8192:
         * stream 40.9 us, tiles 128 x 64 in two parts 22.2) */
        if (form < STREAM ? p.M > 4 * tx : form == STREAM && p.M > 4 * (int64_t)p.N) continue;
        /* parts: as told, at most one a K block; else up to 16 of two blocks or more
         * (of tiles: rows already share K among wavefronts) */
        const int32_t told = std::max(1, std::min({splits, p.nk, 256}));
        for (int32_t s = splits ? told : 1; s <= (splits ? told : form < STREAM ? 1 : 16) && (splits || s == 1 || 2 * s <= p.nk); s *= 2) {
            const double t = time_of(p, form, s, cus);
            if (t < best) {
                best = t;
                p.form = form;
                p.splits = s;
            }
        }
    }
    p.resident = kForms[p.form].resident * cus;
    p.part_planes = planes_of(p, p.form, p.splits);
    p.ldp = ((int64_t)p.N + 3) / 4 * 4;
    p.part = nullptr;
    return std::max(units_of(p, p.form) * p.splits, (((int64_t)p.M + 15) / 16) * (((int64_t)p.N + 127) / 128));
}

namespace {

/* The workgroups of a form whose grid has one each. */
dim3 whole_grid(const BlockGemmParams &p, int32_t form)
{
    const int64_t tx = kForms[form].tx, tn = kForms[form].tw >> p.two;
    return dim3((uint32_t)((p.N + tn - 1) / tn), (uint32_t)((p.M + tx - 1) / tx), (uint32_t)p.splits);
}

template <int FORM, int NW, int ST>
void launch_rows(const BlockGemmParams &p, hipStream_t stream)
{
    constexpr int FX = kForms[FORM].tx / 16, FW = kForms[FORM].tw / 16;
    const dim3 grid = whole_grid(p, FORM), block(NW * 64);
    if (p.two && p.exact)
        hipLaunchKernelGGL((block_rows_kernel<FX, FW, NW, ST, true, true>), grid, block, 0, stream, p);
    else if (p.two)
        hipLaunchKernelGGL((block_rows_kernel<FX, FW, NW, ST, true, false>), grid, block, 0, stream, p);
    else if (p.exact)
        hipLaunchKernelGGL((block_rows_kernel<FX, FW, NW, ST, false, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((block_rows_kernel<FX, FW, NW, ST, false, false>), grid, block, 0, stream, p);
}

void launch_stream(const BlockGemmParams &p, hipStream_t stream)
{
    const dim3 grid = whole_grid(p, STREAM), block(448);
    if (p.two && p.exact)
        hipLaunchKernelGGL((block_stream_kernel<2, 3, 7, true, true>), grid, block, 0, stream, p);
    else if (p.two)
        hipLaunchKernelGGL((block_stream_kernel<2, 3, 7, true, false>), grid, block, 0, stream, p);
    else if (p.exact)
        hipLaunchKernelGGL((block_stream_kernel<2, 3, 7, false, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((block_stream_kernel<2, 3, 7, false, false>), grid, block, 0, stream, p);
}

template <int FORM, int WX, int WW, int ST, int MINB, bool EXACT>
void launch_tile(const BlockGemmParams &p, hipStream_t stream)
{
    constexpr int TX = kForms[FORM].tx, TW = kForms[FORM].tw;
    const int64_t tn = TW >> p.two, units = (((int64_t)p.M + TX - 1) / TX) * ((p.N + tn - 1) / tn) * p.splits;
    const dim3 grid((uint32_t)std::min<int64_t>(units, p.resident)), block(WX * WW * 64);
    if (p.two)
        hipLaunchKernelGGL((block_tile_kernel<TX, TW, WX, WW, ST, MINB, true, EXACT>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((block_tile_kernel<TX, TW, WX, WW, ST, MINB, false, EXACT>), grid, block, 0, stream, p);
}

template <int FORM, int WX, int WW, int ST, int MINB>
void launch_either(const BlockGemmParams &p, hipStream_t stream)
{
    if (p.exact)
        launch_tile<FORM, WX, WW, ST, MINB, true>(p, stream);
    else
        launch_tile<FORM, WX, WW, ST, MINB, false>(p, stream);
}

} /* namespace */

hipError_t launch_block_gemm(const BlockGemmParams &p, hipStream_t stream)
{
    switch (p.form) {
    case ROWS16: launch_rows<ROWS16, 8, 3>(p, stream); break;
    case ROWS16_PAIR: launch_rows<ROWS16_PAIR, 4, 3>(p, stream); break;
    case ROWS32: launch_rows<ROWS32, 4, 2>(p, stream); break;
    case ROWS64: launch_rows<ROWS64, 4, 3>(p, stream); break;
    case ROWS64_PAIR: launch_rows<ROWS64_PAIR, 2, 3>(p, stream); break;
    case STREAM: launch_stream(p, stream); break;
    case TILE_64: launch_either<TILE_64, 2, 2, 6, 1>(p, stream); break;
    case TILE_128: launch_either<TILE_128, 2, 4, 4, 2>(p, stream); break;
    case TILE_128_PAIR: launch_either<TILE_128_PAIR, 2, 2, 2, 2>(p, stream); break;
    case TILE_256: launch_tile<TILE_256, 4, 2, 2, 2, false>(p, stream); break;
    default: launch_either<TILE_WIDE, 2, 4, 3, 2>(p, stream); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.part_planes) return e;
    const int64_t groups = (((int64_t)p.M + 15) / 16) * (((int64_t)p.N + 127) / 128);
    hipLaunchKernelGGL(block_finish_kernel, dim3((uint32_t)groups), dim3(256), 0, stream, p);
    return hipGetLastError();
}

} /* namespace g355 */
