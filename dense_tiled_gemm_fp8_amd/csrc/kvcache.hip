/*
 * kvcache.hip -- keys and values in pages of E4M3 codes, with one E8M0 scale
 * for each page and head, and the attention that reads them.
 *
 *   k [pages][H][page][D]     a token's row of a head is contiguous
 *   v [pages][H][D][page]     a channel's tokens are contiguous, so that the
 *                             second product of attention reads its operand
 *                             in the matrix instruction's order
 *
 *   kv_append_kernel          writes the new tokens of a step, keys rotated by
 *                             their position
 *   attention_kernel          softmax(scale q k^T) v for 16 rows (query token
 *                             and head of one key head) at a time
 *   attention_combine_kernel  joins the parts of a split key axis
 *
 * A page id outside [0, pages) is never followed: its tokens are not written
 * and nothing sees them.
 */
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dma.h"
#include "serve.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
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

/* 2^e for e in [-149, 127]; under 2^-126 it is subnormal. */
__device__ __forceinline__ float pow2(int32_t e) { return __builtin_bit_cast(float, e < -126 ? 1u << (e + 149) : (uint32_t)(e + 127) << 23); }

/* New rows of a sequence: rows [row, row + n), the first at position pos
 * (negative where the sequence is shorter than its rows), length len.  Rows past
 * max_new are left out and leave the others where they are. */
struct Seq {
    int32_t row, n, pos, len;
};

__device__ __forceinline__ Seq sequence(const KvParams &c, int32_t b)
{
    Seq s;
    int32_t rows = c.max_new;
    s.row = b * c.max_new;
    if (c.q_start) {
        s.row = min(max(c.q_start[b], 0), c.tokens);
        rows = min(max(c.q_start[b + 1], s.row), c.tokens) - s.row;
    }
    s.n = min(rows, c.max_new);
    s.len = min(max(c.lens[b], 0), c.max_len);
    s.pos = s.len - rows;
    return s;
}

/* ---------------------------------------------------------------- append */

__device__ __forceinline__ void unpack8(u32x4 a, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = a[j];
        v[2 * j] = __builtin_bit_cast(float, w << 16);
        v[2 * j + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
    }
}

/* a c - b s or, for the second of a pair, a c + b s.  The products of a 16-bit
 * and a 32-bit value are exact in 64 bits, so each result is rounded to 32
 * bits once. */
__device__ __forceinline__ float turned(float a, float b, float c, float s, bool second)
{
    const double bs = (double)b * (double)s;
    return (float)((double)a * (double)c + (second ? bs : -bs));
}

/* 8 values of channels d0 .. d0 + 7 of one token's head at x, rotated for
 * position pos: pairs (a, b) become (a cos - b sin, b cos + a sin). */
__device__ __forceinline__ void rotate8(const KvAppendParams &p, const uint16_t *x, int32_t d0, int32_t pos, float (&v)[8])
{
    const int32_t half = p.rot >> 1;
    const float *cs = p.cos + (int64_t)pos * half, *sn = p.sin + (int64_t)pos * half;
    unpack8(*(const u32x4 *)(x + d0), v);
    if (p.whole) {
        /* 16 channels' pairs or none in each 8: everything by vectors */
        if (d0 >= p.rot) return;
        if (p.interleaved) {
            const f32x4 c = *(const f32x4 *)(cs + d0 / 2), s = *(const f32x4 *)(sn + d0 / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = v[2 * j], b = v[2 * j + 1], cj = c[j], sj = s[j];
                v[2 * j] = turned(a, b, cj, sj, false);
                v[2 * j + 1] = turned(b, a, cj, sj, true);
            }
        } else {
            const bool second = d0 >= half;
            const int32_t i = second ? d0 - half : d0;
            float w[8];
            unpack8(*(const u32x4 *)(x + (second ? i : d0 + half)), w);
            const f32x4 c0 = *(const f32x4 *)(cs + i), c1 = *(const f32x4 *)(cs + i + 4);
            const f32x4 s0 = *(const f32x4 *)(sn + i), s1 = *(const f32x4 *)(sn + i + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ca = c0[j], cb = c1[j], sa = s0[j], sb = s1[j];
                v[j] = turned(v[j], w[j], ca, sa, second);
                v[j + 4] = turned(v[j + 4], w[j + 4], cb, sb, second);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int32_t d = d0 + j;
        if (d >= p.rot) continue;
        const bool second = p.interleaved ? d & 1 : d >= half;
        const int32_t other = p.interleaved ? d ^ 1 : second ? d - half : d + half;
        const int32_t i = p.interleaved ? d >> 1 : second ? d - half : d;
        v[j] = turned(v[j], bf16_value(x[other]), cs[i], sn[i], second);
    }
}

/* E4M3 code pair of two values after the scale; infinities go to the largest
 * value, a NaN stays one. */
__device__ __forceinline__ float saturate(float t) { return fabsf(t) > 448.0f ? __builtin_copysignf(448.0f, t) : t; }

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(a), saturate(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(saturate(c), saturate(d), w, true);
}

/* Four codes decoded, scaled and encoded again. */
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f)
{
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    const float a = lo[0], b = lo[1], c = hi[0], d = hi[1];
    return encode4(a * f, b * f, c * f, d * f);
}

/* Exponent of the smallest power of two that brings a to 448 or under, in
 * [-100, 120]: 448 is 1.75 * 2^8. */
__device__ __forceinline__ int32_t block_exponent(float a)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, a);
    const int32_t e = (int32_t)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, -100), 120);
}

} /* namespace */

/* Work of the append, for sequence blockIdx.y: workgroups 0 .. kv_units - 1 each
 * write the new tokens of one page, head and of keys or values; those behind
 * rotate q, 256 octets of channels each.
 *
 * A page's new tokens stay in registers (ITEMS octets a thread) between finding
 * their largest magnitude and encoding them, so they are read once; values go
 * through LDS as codes to lie along tokens.  What takes the time of a step of
 * single tokens is the chain lengths -> page id -> scale, each a load that
 * waits for the one before: tokens and tables are loaded beside it.
 *
 * Measured: 32 sequences, one token, 32 query and 8 key heads of 128, all of a
 * head rotated: 4.8 us, that chain.  8 x 1000 tokens of 16 and 4 heads: 17.6 us
 * for 77 MB, 4.4 TB/s, where a large copy reaches 4.8 (62 us when tokens were
 * read twice and values written a byte at a time). */
template <int ITEMS>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendParams p, int32_t kv_units)
{
    const KvParams &c = p.c;
    const int32_t D = p.D, oct = D >> 3, oct_log2 = D == 64 ? 3 : D == 128 ? 4 : 5;
    const int32_t b = blockIdx.y;
    const Seq s = sequence(c, b);
    if ((int32_t)blockIdx.x >= kv_units) {
        const uint32_t at = (blockIdx.x - (uint32_t)kv_units) * 256u + threadIdx.x;
        const uint32_t row = at >> oct_log2;           /* token and head           */
        const int32_t i = (int32_t)(row / (uint32_t)p.Hq), head = (int32_t)(row % (uint32_t)p.Hq);
        const int32_t d0 = (int32_t)(at & (uint32_t)(oct - 1)) * 8;
        if (i >= s.n || s.pos + i < 0) return;
        float v[8];
        const uint16_t *x = p.q + (s.row + i) * p.ldq + head * D;
        if (p.rot)
            rotate8(p, x, d0, s.pos + i, v);
        else
            unpack8(*(const u32x4 *)(x + d0), v);
        *(u32x4 *)(p.q_out + (s.row + i) * p.ldqo + head * D + d0) =
            u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        return;
    }
    __shared__ float red[4];
    /* codes of values, by channel: the new tokens' slots from a multiple of 16
     * to one (at most 30 more than there are tokens, of which D times as many as
     * 2048 ITEMS at most), and four bytes that spread channels over the banks */
    __shared__ __align__(16) uint8_t codes[ITEMS * 2048 + 34 * 256];
    const bool keys = (blockIdx.x & 1) == 0;
    const int32_t h = (int32_t)(blockIdx.x >> 1) % c.H, j = (int32_t)(blockIdx.x >> 1) / c.H;
    const int32_t first = max(s.pos, 0);
    const int32_t pg = (first >> c.page_log2) + j, base = pg << c.page_log2;
    const int32_t lo = max(first, base), hi = min(s.pos + s.n, base + c.page);
    if (s.n == 0 || lo >= hi) return;
    const int32_t id = c.table[(int64_t)b * c.table_ld + pg];
    const uint16_t *x = keys ? p.xk + h * D : p.xv + h * D;
    const int64_t ld = keys ? p.ldk : p.ldv;
    const bool turn = keys && p.rot != 0;

    float v[ITEMS][8];
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int32_t w = k * 256 + (int32_t)threadIdx.x, t = lo + (w >> oct_log2), d0 = (w & (oct - 1)) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
        if (t < hi) {
            const uint16_t *row = x + (s.row + t - s.pos) * ld;
            if (turn)
                rotate8(p, row, d0, t, v[k]);
            else
                unpack8(*(const u32x4 *)(row + d0), v[k]);
        }
    }
    if (id < 0 || id >= c.pages) return;
    const int64_t block = (int64_t)id * c.H + h;
    uint8_t *scale = (keys ? c.k_scale : c.v_scale) + block;
    const int32_t e_old = (int32_t)*scale - 127;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[k][i]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    int32_t e = block_exponent(m);
    const bool begins = lo == base;
    if (!begins) e = max(e, e_old);
    const bool grew = !begins && e > e_old;       /* older tokens are rewritten */
    const int32_t ahead = lo - base, upto = hi - base;
    /* e is up to 128 where the page's scale was byte 255 */
    const float down = pow2(-e), older = pow2(max(e_old - e, -60));
    if (threadIdx.x == 0) *scale = (uint8_t)(e + 127);

    uint8_t *out = (keys ? c.k : c.v) + block * c.page * D;
    const int32_t from = ahead & ~15, pitch = ((upto + 15) & ~15) - from + 4;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int32_t w = k * 256 + (int32_t)threadIdx.x, slot = ahead + (w >> oct_log2), d0 = (w & (oct - 1)) * 8;
        if (slot >= upto) continue;
        const uint32_t a = encode4(v[k][0] * down, v[k][1] * down, v[k][2] * down, v[k][3] * down);
        const uint32_t d = encode4(v[k][4] * down, v[k][5] * down, v[k][6] * down, v[k][7] * down);
        if (keys) {
            *(uint2 *)(out + slot * D + d0) = make_uint2(a, d);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                codes[(d0 + i) * pitch + slot - from] = (uint8_t)(a >> (8 * i));
                codes[(d0 + 4 + i) * pitch + slot - from] = (uint8_t)(d >> (8 * i));
            }
        }
    }
    if (keys) {
        if (grew)
            for (int32_t w = threadIdx.x; w < ahead * oct; w += 256) {
                uint2 *at = (uint2 *)(out + w * 8);
                *at = make_uint2(rescale4(at->x, older), rescale4(at->y, older));
            }
        return;
    }
    __syncthreads();
    /* 16 slots of a channel a thread; slots that are not new are read first,
     * where any of the 16 is new or rewritten */
    const int32_t g0 = grew ? 0 : ahead >> 4, groups = ((upto + 15) >> 4) - g0;
    for (int32_t w = threadIdx.x; w < groups * D; w += 256) {
        const int32_t d = w / groups, slot = (g0 + w % groups) * 16;
        u32x4 *at = (u32x4 *)(out + d * c.page + slot);
        u32x4 code = {0, 0, 0, 0};
        if (slot >= from) {
            const uint32_t *mine = (const uint32_t *)(codes + d * pitch + slot - from);
            code = u32x4{mine[0], mine[1], mine[2], mine[3]};
        }
        const int32_t n0 = min(max(ahead - slot, 0), 16), n1 = min(upto - slot, 16);
        if (n0 > 0 || n1 < 16) {
            u32x4 old = *at;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                /* bytes [n0, n1) are new, those under n0 older */
                const uint32_t below0 = n0 >= 4 * i + 4 ? 0xFFFFFFFFu : n0 <= 4 * i ? 0u : (1u << (8 * (n0 - 4 * i))) - 1u;
                const uint32_t below1 = n1 >= 4 * i + 4 ? 0xFFFFFFFFu : n1 <= 4 * i ? 0u : (1u << (8 * (n1 - 4 * i))) - 1u;
                const uint32_t was = old[i], moved = grew ? rescale4(was, older) : was;
                const uint32_t fresh = below1 & ~below0;
                code[i] = (code[i] & fresh) | (moved & below0) | (was & ~(fresh | below0));
            }
        }
        *at = code;
    }
}

namespace {

template <int ITEMS>
void launch_append(const KvAppendParams &p, int32_t kv_units, int32_t q_blocks, hipStream_t stream)
{
    hipLaunchKernelGGL(kv_append_kernel<ITEMS>, dim3((uint32_t)(kv_units + q_blocks), (uint32_t)p.c.B), dim3(256), 0, stream, p, kv_units);
}

} /* namespace */

hipError_t launch_kv_append(const KvAppendParams &p, hipStream_t stream)
{
    /* pages that max_new tokens can touch */
    const int32_t kv_units = ((p.c.max_new + p.c.page - 2) / p.c.page + 1) * p.c.H * 2;
    const int32_t q_blocks = p.q ? (int32_t)(((int64_t)p.c.max_new * p.Hq * (p.D >> 3) + 255) / 256) : 0;
    /* octets of the most new tokens that one page can get, by 256 */
    const int32_t items = (std::min(p.c.max_new, p.c.page) * (p.D >> 3) + 255) / 256;
    if (items <= 1)
        launch_append<1>(p, kv_units, q_blocks, stream);
    else if (items <= 2)
        launch_append<2>(p, kv_units, q_blocks, stream);
    else if (items <= 4)
        launch_append<4>(p, kv_units, q_blocks, stream);
    else if (items <= 8)
        launch_append<8>(p, kv_units, q_blocks, stream);
    else
        launch_append<16>(p, kv_units, q_blocks, stream);
    return hipGetLastError();
}

/* ------------------------------------------------------------- attention */

namespace {

/* What a tile of rows sees: `count` rows from r0 on of a sequence's n * group,
 * the positions of the first and last, and the 64-token chunks to visit (those
 * of the first tokens that stay visible, then the run that ends at the last
 * row's position). */
struct Tile {
    Seq s;
    int32_t rows, pos_lo, pos_hi;
    int32_t sink_chunks, first_chunk, total;
    int32_t parts;                /* splits with work                         */
};

__device__ __forceinline__ Tile row_tile(const AttnParams &p, int32_t b, int32_t r0, int32_t count)
{
    Tile t;
    t.s = sequence(p.c, b);
    t.rows = t.s.n * p.group;
    t.pos_lo = t.s.pos + quotient(r0, p.by_group);
    t.pos_hi = t.s.pos + quotient(max(min(r0 + count - 1, t.rows - 1), 0), p.by_group);
    t.sink_chunks = t.first_chunk = t.total = 0;
    if (r0 < t.rows && t.pos_hi >= 0) {
        if (p.window) {
            t.first_chunk = max(t.pos_lo - p.window + 1, 0) >> 6;
            t.sink_chunks = min((int32_t)(((int64_t)p.sinks + 63) >> 6), t.first_chunk);
        }
        t.total = t.sink_chunks + ((t.pos_hi + 64) >> 6) - t.first_chunk;
    }
    t.parts = min(p.splits, max((t.total + p.part_chunks - 1) / p.part_chunks, 1));
    return t;
}

/* 8 E4M3 codes to bf16, times a power of two (exact). */
__device__ __forceinline__ bf16x8 decode8(uint32_t a, uint32_t b, float s)
{
    bf16x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    return __builtin_bit_cast(bf16x8, v);
}

/* Largest of three (a NaN only if all are); fmaxf would first pass each operand
 * through an instruction of its own to quiet NaNs. */
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

/* Largest over the four lanes of a row (lane / 16), in each of them. */
__device__ __forceinline__ float row_max(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t lo = r[0], hi = r[1];
    const float y = max3(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi), x);
    const uint32_t c = __builtin_bit_cast(uint32_t, y);
    auto t = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    const uint32_t even = t[0], odd = t[1];
    return max3(__builtin_bit_cast(float, even), __builtin_bit_cast(float, odd), y);
}

/* Bits of the 16 tokens from t on that rows at positions lo to hi see between
 * them. */
__device__ __forceinline__ uint32_t seen16(const AttnParams &p, int32_t t, int32_t lo, int32_t hi)
{
    auto below = [](int32_t n) { return (1u << min(max(n, 0), 16)) - 1u; };
    uint32_t bits = below(hi + 1 - t);
    if (p.window) bits &= ~below(lo + 1 - p.window - t) | below(p.sinks - t);
    return bits;
}

/* Four bits to the bytes of a word. */
__device__ __forceinline__ uint32_t bytes_of(uint32_t bits) { return ((bits & 15u) * 0x00204081u & 0x01010101u) * 0xFFu; }

/* Four channels of a row r: bf16 sums over the total weight, and the logarithm
 * of that weight. */
__device__ __forceinline__ void write_out(const AttnParams &p, const Tile &t, int32_t h, int32_t r, int32_t dt, int32_t q, f32x4 sum,
                                          float m, float l)
{
    const int32_t i = quotient(r, p.by_group), head = h * p.group + r - i * p.group;
    const int64_t row = t.s.row + i;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const float a = sum[0] * inv, b = sum[1] * inv, c = sum[2] * inv, d = sum[3] * inv;
    *(uint2 *)(p.o + row * p.ldo + head * p.D + 16 * dt + 4 * q) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
    if (p.lse && dt == 0 && q == 0)
        p.lse[row * p.Hq + head] = l > 0.0f || l != l ? (m + __builtin_log2f(l)) * 0.69314718055994531f : -__builtin_inff();
}

} /* namespace */

/*
 * A workgroup: 16 NR rows of one sequence and key head, one part of their
 * chunks; its NW wavefronts take the chunks (64 tokens) in turn, each with its
 * own running maximum and sum, and join in LDS at the end.
 *
 * Both products run on v_mfma_f32_16x16x32_bf16 with the cache as the first
 * operand: S^T = K Q^T, O^T = V^T P^T.  Lane l is row l % 16 of a row tile in
 * both results and in P^T, so softmax statistics are one value a lane and row
 * tile.  The matrix instruction sums over any order of its 32 values that both
 * operands share, and takes its rows in any order; so product t of a chunk
 * takes as row i = 4a + b the token 16a + 4t + b.  Lane (r, q) then gets the
 * scores of tokens 16q .. 16q + 15, which is the order in which it holds P^T
 * for the second product and takes 16 contiguous tokens of a channel of V:
 * nothing is exchanged between lanes.  Codes become bf16 with the block's power
 * of two in one conversion, exactly.
 *
 * The cache goes straight to LDS, lanes along a token's channels (K) or a
 * channel's tokens (V) so that the memory unit gets its 64 bytes from four
 * neighbours; loads in the matrix order took four times the cycles.  Units of
 * 16 bytes are exchanged within a token's (a channel's) row, so that the
 * reads are free of bank conflicts.  A wavefront has room for one chunk of each:
 * the next chunk's keys are sent off when this one's are read, under the softmax
 * and the second product, its values when that product has read its own; page
 * ids come one chunk further ahead and scales with their pages, all by the same
 * copies, so the waits below count them all and the compiler adds none.
 *
 * Measured: 64 sequences of 4096 to 8192 tokens, 32 query and 8 key heads of 128,
 * one token: 147 us for 811 MB, 5.5 TB/s: memory.  2 x 65536 tokens, 16 and 2
 * heads: 15.5 us for 59 MB, 3.8 TB/s, as all workgroups begin and end together,
 * and 3.8 us for the join of their parts.  One sequence of 700 tokens, 8 heads of
 * 64: 7.5 us, the chain lengths -> page id -> codes -> two products
 * twice over, and the join.  4 x 512 new tokens of 16 and 4 heads of 128 with a
 * window of 2048: 54 us, 0.52 PFLOP/s; of a SIMD's cycles half go to vector
 * instructions (conversions of codes and exponentials, in equal parts) and a
 * quarter to matrix instructions, and two wavefronts do not hide all of each
 * other's waits.
 */
template <int D, int NR, int NW>
__global__ __launch_bounds__(NW * 64, NR == 2 && D <= 128 ? 2 : 1) void attention_kernel(AttnParams p)
{
    constexpr int DT = D / 16, DS = D / 32, DL = D / 64, UNITS = D / 16;
    const KvParams &c = p.c;
    const int32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t lr = lane & 15, q = lane >> 4;
    /* Workgroups go to the eight dies in turn, each with its own L2: where a
     * sequence and head has several row tiles, they go to one die, which then
     * reads its tokens once (4096 new tokens of 32 heads of 128: 246 us without,
     * 216 so).  The last rows see the most tokens and begin first (262 us the
     * other way round). */
    int32_t part = blockIdx.x, tile = blockIdx.y, pair = blockIdx.z;
    if (p.row_tiles > 1) {
        if (c.B * c.H % 8 == 0) {
            const uint32_t splits = (uint32_t)p.splits, each = splits * (uint32_t)p.row_tiles;
            const uint64_t at = ((uint64_t)each * blockIdx.z + splits * blockIdx.y + blockIdx.x) >> 3;
            const uint32_t turn = (uint32_t)(at / each), rest = (uint32_t)(at - (uint64_t)turn * each);
            pair = (int32_t)(8 * turn + ((splits * blockIdx.y + blockIdx.x + each * blockIdx.z) & 7));
            tile = (int32_t)(rest / splits);
            part = (int32_t)(rest % splits);
        }
        tile = p.row_tiles - 1 - tile;
    }
    const int32_t b = pair / c.H, h = pair % c.H, r0 = tile * (16 * NR);
    const Tile t = row_tile(p, b, r0, 16 * NR);
    if (r0 >= t.rows || part >= t.parts) return;
    int32_t begin = 0, end = t.total;
    if (t.parts > 1) {
        begin = (int32_t)((int64_t)t.total * part / t.parts);
        end = (int32_t)((int64_t)t.total * (part + 1) / t.parts);
    }

    /* LDS of a wavefront: a chunk of keys, one of values, page ids of two
     * chunks, scales of a chunk's key and value pages; behind the loop the
     * sums to join */
    constexpr int KB = 64 * D, OWN = 2 * KB + 4 * 256;
    static_assert(NR * DT * 1024 <= OWN, "sums of a wavefront take the place of its chunk");
    __shared__ __align__(16) uint8_t store[NW * OWN];
    __shared__ float st[NW][2][16 * NR];
    const uint32_t base = __builtin_amdgcn_readfirstlane(lds_addr(store) + wave * OWN);
    uint8_t *own = store + wave * OWN;

    int32_t pos[NR];
    bf16x8 qf[NR][DS];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int32_t r = min(r0 + 16 * i + lr, t.rows - 1);
        const int32_t token = quotient(r, p.by_group);
        pos[i] = t.s.pos + token;
        const uint16_t *row = p.q + (int64_t)(t.s.row + token) * p.ldq + (h * p.group + r - token * p.group) * D + q * (D / 4);
#pragma unroll
        for (int x = 0; x < DS; ++x) qf[i][x] = __builtin_bit_cast(bf16x8, *(const u32x4 *)(row + 8 * x));
    }

    f32x4 o[NR][DT], lw[NR];                      /* lw: sum of the weights as the second product takes them */
    float m[NR], l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i] = -__builtin_inff();
        l[i] = 0.0f;
        lw[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < DT; ++x) o[i][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    /* 16-token blocks: of the chunk's four, the one of the lane's key rows
     * (ksub), of its scores and values (q), and that its copies of values take
     * (vsub; lane i < 4 has block i) */
    const int32_t ksub = lr >> 2, vsub = (lane & 3) ^ q;
    const int32_t *table = c.table + (int64_t)b * c.table_ld;
    auto token0 = [&](int32_t it) __attribute__((always_inline)) {
        return (it < t.sink_chunks ? it : t.first_chunk + it - t.sink_chunks) << 6;
    };
    /* copies of keys: unit `lane % UNITS` of a row takes the piece that is
     * exchanged into it, by the token's low bits and its block */
    const int32_t krow = lane / UNITS;
    uint32_t key_at[DL];
#pragma unroll
    for (int y = 0; y < DL; ++y) {
        const int32_t tk = y * (64 / UNITS) + krow;
        const int32_t swap = D == 64 ? 0 : D == 128 ? tk >> 1 & 1 : tk & 3;
        key_at[y] = (uint32_t)(tk * D + ((lane % UNITS) ^ swap) * 16);
    }
    constexpr int BLOCK_BITS = D == 64 ? 4 : D == 128 ? 5 : 6;

    auto copy_ids = [&](int32_t half, int32_t it) __attribute__((always_inline)) {
        const int32_t tk = min(token0(min(it, end - 1)) + 16 * vsub, t.s.len - 1);
        dma_global4(base + 2 * KB + half * 256, table + (tk >> c.page_log2));
    };
    /* page id of the copies' block, 0 in place of one that is no page (its
     * tokens are masked); `all` of the lane's blocks are pages of tokens held */
    auto ids_of = [&](int32_t half, int32_t t0, int32_t &id, bool &kok, bool &vok) __attribute__((always_inline)) {
        const int32_t *ids = (const int32_t *)(own + 2 * KB + half * 256);
        const int32_t v = ids[lane], kid = ids[ksub], vid = ids[q];
        id = v >= 0 && v < c.pages ? v : 0;
        kok = kid >= 0 && kid < c.pages && t0 + 16 * ksub < t.s.len;
        vok = vid >= 0 && vid < c.pages && t0 + 16 * q < t.s.len;
    };
    auto copy_keys = [&](int32_t id, int32_t t0) __attribute__((always_inline)) {
        dma_global1(base + 2 * KB + 512, c.k_scale + ((int64_t)id * c.H + h));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t block = (int64_t)__builtin_amdgcn_readlane(id, x) * c.H + h;
            const uint8_t *at = c.k + (block * c.page + ((t0 + 16 * x) & (c.page - 1))) * D;
#pragma unroll
            for (int y = 0; y < DL; ++y) dma_global16(base + (x * DL + y) * 1024, at + (key_at[y] ^ (uint32_t)(x << BLOCK_BITS)));
        }
    };
    auto copy_values = [&](int32_t id, int32_t t0) __attribute__((always_inline)) {
        const int64_t block = (int64_t)id * c.H + h;
        dma_global1(base + 2 * KB + 768, c.v_scale + block);
        const uint8_t *at = c.v + (block * D + (lane >> 2)) * c.page + ((t0 + 16 * vsub) & (c.page - 1));
#pragma unroll
        for (int x = 0; x < DT; ++x) dma_global16(base + KB + x * 1024, at + 16 * x * c.page);
    };
    constexpr int KEYS = 2 + 4 * DL, VALUES = 1 + DT;   /* copies sent together */
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

    int32_t it = begin + wave;
    if (it < end) {
        int32_t t0 = token0(it), id, half = 0;
        bool kok, vok;
        copy_ids(0, it);
        wait_vmcnt<0>();
        ids_of(0, t0, id, kok, vok);
        copy_ids(1, it + NW);
        copy_keys(id, t0);
        copy_values(id, t0);
#pragma unroll 1
        for (; it < end; it += NW) {
            const int32_t vt = t0 + 16 * q;

            wait_vmcnt<VALUES>();
            const float ks = __builtin_bit_cast(float, *(const uint32_t *)(own + 2 * KB + 512 + 4 * ksub) << 23);
            f32x4 s[NR][4];
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[i][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int y = 0; y < DL; ++y) {
                /* products before the other wavefront's softmax (3 % of the time
                 * of prompts; for heads of 256 a loss of 3 %) */
                if constexpr (NR == 2 && D <= 128) __builtin_amdgcn_s_setprio(1);
                u32x4 kr[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int32_t tk = 16 * ksub + 4 * x + (lr & 3);
                    const int32_t swap = D == 64 ? ksub : D == 128 ? (tk >> 1 & 1) | ksub << 1 : (tk & 3) | ksub << 2;
                    kr[x] = *(const u32x4 *)(own + tk * D + (((q * DL + y) ^ swap) << 4));
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    bf16x8 kf[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) kf[x] = decode8(kr[x][2 * z], kr[x][2 * z + 1], ks);
#pragma unroll
                    for (int i = 0; i < NR; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s[i][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[x], qf[i][2 * y + z], s[i][x], 0, 0, 0);
                }
            }
            if constexpr (NR == 2 && D <= 128) __builtin_amdgcn_s_setprio(0);
            /* this chunk's keys are read: the next one's, and ids after that */
            const int32_t t1 = token0(min(it + NW, end - 1));
            int32_t id1;
            bool kok1, vok1;
            ids_of(half ^ 1, t1, id1, kok1, vok1);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            copy_ids(half, it + 2 * NW);
            copy_keys(id1, t1);

            /* every row sees every token of the chunk, or masks */
            const bool inside = t0 + 63 <= t.pos_lo && (!p.window || t0 > t.pos_hi - p.window || t0 + 63 < p.sinks);
            if (!inside || __ballot(!(kok && vok)) != 0) {
                uint32_t mine[NR];                /* tokens that the lane's rows see    */
#pragma unroll
                for (int i = 0; i < NR; ++i) mine[i] = vok ? seen16(p, vt, pos[i], pos[i]) : 0u;
                /* those that some row sees: up to the last row's position,
                 * within the first row's window */
                const uint32_t some_row = vok ? seen16(p, vt, t.pos_lo, t.pos_hi) : 0u;
                uint32_t any[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) any[y] = bytes_of(some_row >> (4 * y));
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int x = 0; x < 16; ++x) s[i][x >> 2][x & 3] = mine[i] >> x & 1u ? s[i][x >> 2][x & 3] : -__builtin_inff();
                /* tokens that no row sees may hold anything, a NaN too, which
                 * a weight of zero would not keep out of the sums: their bytes
                 * are cleared (a lane clears what it reads itself), and so is
                 * the scale of a block that no row sees (0 under byte 255 is a
                 * NaN).  A value that some of the rows see is not finite, and
                 * found as a NaN, if its code is one, if its block's scale is
                 * (byte 255), or if it is 2^128 or more, the code of 2^k being
                 * 8 (k + 7): bit 7 of the code plus 128 - `past`. */
                wait_vmcnt<KEYS>();
                uint32_t *vbyte = (uint32_t *)(own + 2 * KB + 768 + 4 * q);
                const uint32_t byte = *vbyte, past = byte == 255 ? 0 : min((262 - byte) << 3, 0x7Fu);
                const uint32_t add = (128 - past) * 0x01010101u;
                if (some_row == 0 || byte == 255) *vbyte = 127;
                u32x4 *mem = (u32x4 *)(own + KB) + lr * 4 + (q ^ (lr >> 2));
                uint32_t nan[4] = {0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < DT; ++x) {
                    u32x4 v = mem[x * 64];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        v[y] &= any[y];
                        nan[y] |= (v[y] & 0x7F7F7F7Fu) + add;
                    }
                    mem[x * 64] = v;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) nan[y] &= any[y];
                const uint32_t some = (nan[0] | nan[1] | nan[2] | nan[3]) & 0x80808080u;
                if (__ballot(some != 0) != 0) {
                    /* what is not finite and seen by some of the rows: out of
                     * the values, and a NaN into the scores of those rows */
                    uint32_t tok = 0;
#pragma unroll
                    for (int x = 0; x < 16; ++x) tok |= (nan[x >> 2] >> (8 * (x & 3) + 7) & 1u) << x;
                    for (int off = 1; off < 16; off <<= 1) tok |= __shfl_xor(tok, off, 64);
                    uint32_t clean[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        if (!(tok >> x & 1u)) clean[x >> 2] |= 0xFFu << (8 * (x & 3));
#pragma unroll
                        for (int i = 0; i < NR; ++i)
                            if ((tok & mine[i]) >> x & 1u) s[i][x >> 2][x & 3] = __builtin_nanf("");
                    }
#pragma unroll
                    for (int x = 0; x < DT; ++x) {
                        u32x4 v = mem[x * 64];
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] &= clean[y];
                        mem[x * 64] = v;
                    }
                }
            }

            bf16x8 pf[NR][2];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                float top = s[i][0][0];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top = max3(top, s[i][x][0], s[i][x][1]);
                    top = max3(top, s[i][x][2], s[i][x][3]);
                }
                top = row_max(top);
                /* the reference of a row's weights moves only when its maximum
                 * has passed it by a factor of 2^8, and then to 2^8 above that
                 * maximum: weights stay under 2^8, and the sums are rarely
                 * touched.  Each row by itself (the others' sums are multiplied
                 * by 1), so that no row's bits depend on another's scores.
                 * Moved to the maximum itself, rows move more often than they did
                 * together: 4 x 512 tokens with a window, heads of 64, 41.7 us
                 * against 40.4, heads of 128 60.8 and 58.8 */
                const float now = fmaxf(m[i], top * p.scale_log2);
                const bool moves = now > m[i] + 8.0f;
                float ref = m[i] == -__builtin_inff() ? 0.0f : m[i];       /* no token seen yet */
                if (__ballot(moves) != 0) {
                    if (moves) ref = now + 8.0f;
                    const float fade = __builtin_amdgcn_exp2f(m[i] - ref);
                    l[i] *= fade;
                    lw[i][0] *= fade;
#pragma unroll
                    for (int x = 0; x < DT; ++x)
#pragma unroll
                        for (int y = 0; y < 4; ++y) o[i][x][y] *= fade;
                    if (moves) m[i] = ref;
                }
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][x][y], p.scale_log2, -ref));
                        s[i][x][y] = e;
                        sum += e;
                    }
                l[i] += sum;
                /* weights enter the second product in 16 bits: each is off by up
                 * to 2^-8 of itself, independently */
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    pf[i][x] = __builtin_bit_cast(bf16x8, u32x4{pack_bf16(s[i][2 * x][0], s[i][2 * x][1]),
                                                                pack_bf16(s[i][2 * x][2], s[i][2 * x][3]),
                                                                pack_bf16(s[i][2 * x + 1][0], s[i][2 * x + 1][1]),
                                                                pack_bf16(s[i][2 * x + 1][2], s[i][2 * x + 1][3])});
            }
            wait_vmcnt<KEYS>();
            const float vs = __builtin_bit_cast(float, *(const uint32_t *)(own + 2 * KB + 768 + 4 * q) << 23);
            if constexpr (NR == 2 && D <= 128) __builtin_amdgcn_s_setprio(1);
            const u32x4 *vals = (const u32x4 *)(own + KB) + lr * 4 + (q ^ (lr >> 2));
            /* the sum of the weights as rounded: what divides the other sums,
             * so that errors they have in common (all, where one token has most
             * of the weight) go out.  Off 64 bits by 0.0017 of the output's
             * size for 700 tokens, which is rounding the output, where dividing
             * by the sum of the unrounded weights is off by 0.0024 */
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < NR; ++i) lw[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pf[i][x], lw[i], 0, 0, 0);
#pragma unroll
            for (int x = 0; x < DT; ++x) {
                const u32x4 v = vals[x * 64];
                const bf16x8 v0 = decode8(v[0], v[1], vs), v1 = decode8(v[2], v[3], vs);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    o[i][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pf[i][0], o[i][x], 0, 0, 0);
                    o[i][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pf[i][1], o[i][x], 0, 0, 0);
                }
            }
            if constexpr (NR == 2 && D <= 128) __builtin_amdgcn_s_setprio(0);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            copy_values(id1, t1);
            t0 = t1;
            kok = kok1;
            vok = vok1;
            half ^= 1;
        }
        wait_vmcnt<0>();                           /* the copies past the end  */
    }

    /* join the wavefronts: statistics of all, then their sums, brought to one
     * reference, each wavefront adding up and storing 16 channels in turn */
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        l[i] += __shfl_xor(l[i], 16, 64);
        l[i] += __shfl_xor(l[i], 32, 64);
        if (q == 0) {
            st[wave][0][16 * i + lr] = m[i];
            st[wave][1][16 * i + lr] = l[i];
        }
    }
    __syncthreads();
    float all[NR], total[NR];
    f32x4 *sums = (f32x4 *)store;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        all[i] = -__builtin_inff();
        total[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) all[i] = fmaxf(all[i], st[w][0][16 * i + lr]);
        const float ref = all[i] == -__builtin_inff() ? 0.0f : all[i];
#pragma unroll
        for (int w = 0; w < NW; ++w) total[i] += st[w][1][16 * i + lr] * __builtin_amdgcn_exp2f(st[w][0][16 * i + lr] - ref);
        /* sums over the rounded weights go on as sums over the others */
        const float mine = lw[i][0], f = __builtin_amdgcn_exp2f(m[i] - ref) * (mine > 0.0f || mine != mine ? l[i] / mine : 1.0f);
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            f32x4 v = o[i][x];
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] *= f;
            sums[((wave * NR + i) * DT + x) * 64 + lane] = v;
        }
    }
    __syncthreads();
    const int64_t slot = (((int64_t)pair * p.row_tiles + tile) * p.splits + part) * NR;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int32_t r = r0 + 16 * i + lr;
        if (r >= t.rows) continue;
        for (int32_t x = wave; x < DT; x += NW) {
            f32x4 v = sums[(i * DT + x) * 64 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += sums[((w * NR + i) * DT + x) * 64 + lane];
            if (t.parts > 1)
                *(f32x4 *)(p.part + ((slot + i) * DT + x) * 256 + lane * 4) = v;
            else
                write_out(p, t, h, r, x, q, v, all[i], total[i]);
        }
        if (t.parts > 1 && q == 0 && wave == 0) {
            p.stat[(slot + i) * 32 + lr] = all[i];
            p.stat[(slot + i) * 32 + 16 + lr] = total[i];
        }
    }
}

/* Joins the parts of 16 rows and 16 channels: eight wavefronts take the parts in
 * turn, eight at a time (all loads of 64 parts in flight at once), and their sums
 * are added in LDS in a fixed order.  Latency bounds it: 64 parts of 4 row tiles
 * of 128 channels, 2.1 MB, in 3.8 us, as long as an empty launch. */
constexpr int kJoinWaves = 8, kJoinParts = 8;

template <int D, int NR>
__global__ __launch_bounds__(kJoinWaves * 64) void attention_combine_kernel(AttnParams p)
{
    constexpr int DT = D / 16;
    const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, q = lane >> 4;
    const int32_t x = blockIdx.x % DT, i = blockIdx.x / DT % NR, tile = blockIdx.x / (DT * NR);
    const int32_t b = blockIdx.y / p.c.H, h = blockIdx.y % p.c.H, r0 = tile * (16 * NR);
    const Tile t = row_tile(p, b, r0, 16 * NR);
    if (r0 + 16 * i >= t.rows || t.parts == 1) return;
    const int32_t r = r0 + 16 * i + lr;
    const int64_t slot = ((int64_t)blockIdx.y * p.row_tiles + tile) * p.splits;
    const float *stat = p.stat + (slot * NR + i) * 32 + lr;
    const float *part = p.part + ((slot * NR + i) * DT + x) * 256 + lane * 4;
    const bool in = r < t.rows;
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t k = wave; k < t.parts; k += kJoinWaves * kJoinParts) {
        float pm[kJoinParts], pl[kJoinParts];
        f32x4 v[kJoinParts];
#pragma unroll
        for (int y = 0; y < kJoinParts; ++y) {
            const int32_t i2 = k + kJoinWaves * y;
            pm[y] = -__builtin_inff();
            pl[y] = 0.0f;
            v[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (in && i2 < t.parts) {
                pm[y] = stat[(int64_t)i2 * NR * 32];
                pl[y] = stat[(int64_t)i2 * NR * 32 + 16];
                v[y] = *(const f32x4 *)(part + (int64_t)i2 * NR * DT * 256);
            }
        }
        float now = m;
#pragma unroll
        for (int y = 0; y < kJoinParts; ++y) now = fmaxf(now, pm[y]);
        const float ref = now == -__builtin_inff() ? 0.0f : now;
        const float fade = __builtin_amdgcn_exp2f(m - ref);
        m = now;
        l *= fade;
#pragma unroll
        for (int z = 0; z < 4; ++z) sum[z] *= fade;
#pragma unroll
        for (int y = 0; y < kJoinParts; ++y) {
            const float f = __builtin_amdgcn_exp2f(pm[y] - ref);
            l += f * pl[y];
#pragma unroll
            for (int z = 0; z < 4; ++z) sum[z] += f * v[y][z];
        }
    }
    __shared__ float st[kJoinWaves][2][64];
    __shared__ f32x4 sums[kJoinWaves][64];
    st[wave][0][lane] = m;
    st[wave][1][lane] = l;
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || !in) return;
    float all = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) all = fmaxf(all, st[w][0][lane]);
    const float ref = all == -__builtin_inff() ? 0.0f : all;
    float total = 0.0f;
    f32x4 out = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(st[w][0][lane] - ref);
        const f32x4 v = sums[w][lane];
        total += f * st[w][1][lane];
#pragma unroll
        for (int z = 0; z < 4; ++z) out[z] += f * v[z];
    }
    write_out(p, t, h, r, x, q, out, all, total);
}

namespace {

template <int D, int NR, int NW>
hipError_t launch_tile(const AttnParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL((attention_kernel<D, NR, NW>), dim3((uint32_t)p.splits, (uint32_t)p.row_tiles, (uint32_t)(p.c.B * p.c.H)),
                       dim3(NW * 64), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((attention_combine_kernel<D, NR>), dim3((uint32_t)(p.row_tiles * NR * (D / 16)), (uint32_t)(p.c.B * p.c.H)),
                       dim3(kJoinWaves * 64), 0, stream, p);
    return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const AttnParams &p, hipStream_t stream)
{
    if (p.tile_rows > 16) {
        if constexpr (D <= 128)
            if (p.waves == 4) return launch_tile<D, 2, 4>(p, stream);
        if (p.waves == 2) return launch_tile<D, 2, 2>(p, stream);
        return hipErrorInvalidValue;
    }
    if constexpr (D <= 128)
        if (p.waves == 8) return launch_tile<D, 1, 8>(p, stream);
    if constexpr (D >= 128)
        if (p.waves == 4) return launch_tile<D, 1, 4>(p, stream);
    if constexpr (D == 256)
        if (p.waves == 2) return launch_tile<D, 1, 2>(p, stream);
    return hipErrorInvalidValue;
}

} /* namespace */

hipError_t launch_attention(const AttnParams &p, hipStream_t stream)
{
    if (p.D == 64) return launch_dim<64>(p, stream);
    if (p.D == 128) return launch_dim<128>(p, stream);
    return launch_dim<256>(p, stream);
}

} /* namespace g355 */
