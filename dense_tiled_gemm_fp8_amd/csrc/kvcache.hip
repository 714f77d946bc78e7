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

#include "serve.h"

namespace g355 {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_value(uint32_t h) { return __builtin_bit_cast(float, h << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float pow2(int32_t e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

/* New rows of a sequence: rows [row, row + n), the first at position pos
 * (negative where the sequence is shorter than its rows), length len. */
struct Seq {
    int32_t row, n, pos, len;
};

__device__ __forceinline__ Seq sequence(const KvParams &c, int32_t b)
{
    Seq s;
    if (c.q_start) {
        const int32_t a = min(max(c.q_start[b], 0), c.tokens);
        const int32_t e = min(max(c.q_start[b + 1], a), c.tokens);
        s.row = a;
        s.n = min(e - a, c.max_new);
    } else {
        s.row = b * c.max_new;
        s.n = c.max_new;
    }
    s.len = min(max(c.lens[b], 0), c.max_len);
    s.pos = s.len - s.n;
    return s;
}

/* ---------------------------------------------------------------- append */

/* 8 values of channels d0 .. d0 + 7 of one token's head at x, rotated for
 * position pos: pairs (a, b) become (a cos - b sin, b cos + a sin).  The
 * products of a 16-bit and a 32-bit value are exact in 64 bits, so each
 * result is rounded to 32 bits once. */
__device__ __forceinline__ void rotate8(const KvAppendParams &p, const uint16_t *x, int32_t d0, int32_t pos, float (&v)[8])
{
    const int32_t half = p.rot >> 1;
    const float *cs = p.cos + (int64_t)pos * half, *sn = p.sin + (int64_t)pos * half;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int32_t d = d0 + j;
        const double a = bf16_value(x[d]);
        if (d >= p.rot) {
            v[j] = (float)a;
        } else {
            int32_t other, i;
            bool second;
            if (p.interleaved) {
                second = d & 1;
                other = d ^ 1;
                i = d >> 1;
            } else {
                second = d >= half;
                other = second ? d - half : d + half;
                i = second ? d - half : d;
            }
            const double b = bf16_value(x[other]);
            const double c = cs[i], s = sn[i];
            v[j] = (float)(second ? a * c + b * s : a * c - b * s);
        }
    }
}

__device__ __forceinline__ void plain8(const uint16_t *x, int32_t d0, float (&v)[8])
{
    const uint4 a = *(const uint4 *)(x + d0);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
        v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
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

/* One workgroup for the new tokens of one page, head and of keys or values
 * (reads them twice: for their largest magnitude, then to write codes); the
 * workgroups behind those rotate q. */
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendParams p, int32_t pages_each, int32_t kv_units, int32_t q_blocks)
{
    const KvParams &c = p.c;
    const int32_t D = p.D, oct = D >> 3;
    if ((int32_t)blockIdx.x >= kv_units) {
        const int32_t u = (int32_t)blockIdx.x - kv_units;
        const Seq s = sequence(c, u / q_blocks);
        const int64_t at = (int64_t)(u % q_blocks) * 256 + threadIdx.x;
        const int32_t per = p.Hq * oct;
        const int32_t i = (int32_t)(at / per), rest = (int32_t)(at % per);
        if (i >= s.n || s.pos + i < 0) return;
        const int32_t head = rest / oct, d0 = rest % oct * 8;
        float v[8];
        const uint16_t *x = p.q + (s.row + i) * p.ldq + head * D;
        if (p.rot)
            rotate8(p, x, d0, s.pos + i, v);
        else
            plain8(x, d0, v);
        *(uint4 *)(p.q_out + (s.row + i) * p.ldqo + head * D + d0) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        return;
    }
    __shared__ float red[4];
    int32_t u = blockIdx.x;
    const bool keys = (u & 1) == 0;
    u >>= 1;
    const int32_t h = u % c.H;
    u /= c.H;
    const int32_t j = u % pages_each, b = u / pages_each;
    const Seq s = sequence(c, b);
    const int32_t first = max(s.pos, 0);
    const int32_t pg = (first >> c.page_log2) + j, base = pg << c.page_log2;
    const int32_t lo = max(first, base), hi = min(s.len, base + c.page);
    if (s.n == 0 || lo >= hi) return;
    const int32_t id = c.table[(int64_t)b * c.table_ld + pg];
    if (id < 0 || id >= c.pages) return;
    const int64_t block = (int64_t)id * c.H + h;
    uint8_t *scale = (keys ? c.k_scale : c.v_scale) + block;
    const int32_t e_old = (int32_t)*scale - 127;
    const uint16_t *x = keys ? p.xk + h * D : p.xv + h * D;
    const int64_t ld = keys ? p.ldk : p.ldv;
    const bool turn = keys && p.rot != 0;
    const int32_t count = hi - lo;

    float m = 0.0f;
    for (int32_t w = threadIdx.x; w < count * oct; w += 256) {
        const int32_t t = lo + w / oct, d0 = w % oct * 8;
        const uint16_t *row = x + (s.row + t - s.pos) * ld;
        float v[8];
        if (turn)
            rotate8(p, row, d0, t, v);
        else
            plain8(row, d0, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    int32_t e = block_exponent(m);
    const bool begins = lo == base;
    if (!begins) e = max(e, e_old);
    /* the block's older tokens, where its scale grew */
    const int32_t from = !begins && e > e_old ? 0 : lo - base;
    const float down = pow2(-e), older = pow2(max(e_old - e, -60));
    if (threadIdx.x == 0) *scale = (uint8_t)(e + 127);

    if (keys) {
        uint8_t *out = c.k + block * c.page * D;
        for (int32_t w = threadIdx.x; w < (hi - base - from) * oct; w += 256) {
            const int32_t slot = from + w / oct, d0 = w % oct * 8;
            uint2 *at = (uint2 *)(out + slot * D + d0);
            uint2 code;
            if (base + slot < lo) {
                code = *at;
                code = make_uint2(rescale4(code.x, older), rescale4(code.y, older));
            } else {
                const uint16_t *row = x + (s.row + base + slot - s.pos) * ld;
                float v[8];
                if (turn)
                    rotate8(p, row, d0, base + slot, v);
                else
                    plain8(row, d0, v);
                code = make_uint2(encode4(v[0] * down, v[1] * down, v[2] * down, v[3] * down),
                                  encode4(v[4] * down, v[5] * down, v[6] * down, v[7] * down));
            }
            *at = code;
        }
    } else {
        /* a thread owns four slots of one channel */
        uint8_t *out = c.v + block * c.page * D;
        const int32_t w0 = from >> 2, words = ((hi - base + 3) >> 2) - w0;
        for (int32_t w = threadIdx.x; w < words * D; w += 256) {
            const int32_t slot = (w0 + w / D) * 4, d = w % D;
            uint32_t *at = (uint32_t *)(out + d * c.page + slot);
            const bool whole = base + slot >= lo && base + slot + 4 <= hi;
            uint32_t code = whole ? 0 : *at;
            if (from == 0 && !begins && !whole) {
                const uint32_t moved = rescale4(code, older);
                const int32_t keep = min(max(lo - base - slot, 0), 4);
                const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
                code = (moved & mask) | (code & ~mask);
            }
            float f[4];
            uint32_t mask = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t t = base + slot + i;
                f[i] = 0.0f;
                if (t >= lo && t < hi) {
                    f[i] = bf16_value(x[(s.row + t - s.pos) * ld + d]) * down;
                    mask |= 0xFFu << (8 * i);
                }
            }
            *at = (encode4(f[0], f[1], f[2], f[3]) & mask) | (code & ~mask);
        }
    }
}

hipError_t launch_kv_append(const KvAppendParams &p, hipStream_t stream)
{
    /* pages that max_new tokens can touch */
    const int32_t pages_each = (p.c.max_new + p.c.page - 2) / p.c.page + 1;
    const int32_t kv_units = p.c.B * pages_each * p.c.H * 2;
    const int64_t per_seq = (int64_t)p.c.max_new * p.Hq * (p.D >> 3);
    const int32_t q_blocks = p.q ? (int32_t)((per_seq + 255) / 256) : 0;
    hipLaunchKernelGGL(kv_append_kernel, dim3((uint32_t)(kv_units + p.c.B * q_blocks)), dim3(256), 0, stream, p, pages_each,
                       kv_units, q_blocks);
    return hipGetLastError();
}

/* ------------------------------------------------------------- attention */

namespace {

/* What a tile of rows sees: rows r0 .. r0 + 15 of a sequence's n * group, the
 * positions of the first and last, and the 64-token chunks to visit (those of
 * the first tokens that stay visible, then the run that ends at the last
 * row's position). */
struct Tile {
    Seq s;
    int32_t rows, pos_lo, pos_hi;
    int32_t sink_chunks, first_chunk, total;
    int32_t parts;                /* splits with work                         */
};

constexpr int kAttnWaves = 4;

__device__ __forceinline__ Tile row_tile(const AttnParams &p, int32_t b, int32_t r0)
{
    Tile t;
    t.s = sequence(p.c, b);
    t.rows = t.s.n * p.group;
    t.pos_lo = t.s.pos + r0 / p.group;
    t.pos_hi = t.s.pos + min(r0 + 15, t.rows - 1) / p.group;
    t.sink_chunks = t.first_chunk = t.total = 0;
    if (r0 < t.rows && t.pos_hi >= 0) {
        if (p.window) {
            t.first_chunk = max(t.pos_lo - p.window + 1, 0) >> 6;
            t.sink_chunks = min((int32_t)(((int64_t)p.sinks + 63) >> 6), t.first_chunk);
        }
        t.total = t.sink_chunks + ((t.pos_hi + 64) >> 6) - t.first_chunk;
    }
    t.parts = min(p.splits, max((t.total + kAttnWaves - 1) / kAttnWaves, 1));
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

/* Output row of a tile's row r: bf16 sums over the total weight, and the
 * logarithm of that weight. */
template <int D>
__device__ __forceinline__ void write_out(const AttnParams &p, const Tile &t, int32_t h, int32_t r, int32_t dt, int32_t q, f32x4 sum,
                                          float m, float l)
{
    const int32_t i = r / p.group, head = h * p.group + r % p.group;
    const int64_t row = t.s.row + i;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const float a = sum[0] * inv, b = sum[1] * inv, c = sum[2] * inv, d = sum[3] * inv;
    *(uint2 *)(p.o + row * p.ldo + head * D + 16 * dt + 4 * q) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
    if (p.lse && dt == 0 && q == 0)
        p.lse[row * p.Hq + head] = l > 0.0f || l != l ? (m + __builtin_log2f(l)) * 0.69314718055994531f : -__builtin_inff();
}

} /* namespace */

/*
 * A workgroup: 16 rows of one sequence and key head, one part of their
 * chunks; its wavefronts take the chunks (64 tokens) in turn, each with its
 * own running maximum and sum, and join in LDS at the end.
 *
 * Both products run on v_mfma_f32_16x16x32_bf16 with the cache as the first
 * operand: S^T = K Q^T, O^T = V^T P^T.  Lane l is row r = l % 16 of the tile
 * in both results and in P^T, so softmax statistics are one value a lane.
 * The matrix instruction sums over any order of its 32 values that both
 * operands share, and takes its rows in any order; so product t of a chunk
 * takes as row i = 4a + b the token 16a + 4t + b.  Lane (r, q) then gets the
 * scores of tokens 16q .. 16q + 15, which is the order in which it holds P^T
 * for the second product and loads 16 contiguous tokens of a channel of V:
 * nothing is exchanged between lanes.  A lane's D / 4 channels of a key row are
 * contiguous as well.  Codes become bf16 with the block's power of two
 * in one conversion, exactly.
 */
template <int D>
__global__ __launch_bounds__(kAttnWaves * 64) void attention_kernel(AttnParams p)
{
    constexpr int DT = D / 16, DS = D / 32, DL = D / 64;
    const KvParams &c = p.c;
    const int32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t lr = lane & 15, q = lane >> 4;
    const int32_t b = blockIdx.z / c.H, h = blockIdx.z % c.H, r0 = blockIdx.y * 16;
    const Tile t = row_tile(p, b, r0);
    if (r0 >= t.rows || (int32_t)blockIdx.x >= t.parts) return;
    const int32_t begin = (int32_t)((int64_t)t.total * blockIdx.x / t.parts);
    const int32_t end = (int32_t)((int64_t)t.total * (blockIdx.x + 1) / t.parts);

    const int32_t r = min(r0 + lr, t.rows - 1);
    const int32_t pos = t.s.pos + r / p.group;
    const uint16_t *qrow = p.q + (int64_t)(t.s.row + r / p.group) * p.ldq + (h * p.group + r % p.group) * D + q * (D / 4);
    bf16x8 qf[DS];
#pragma unroll
    for (int i = 0; i < DS; ++i) qf[i] = __builtin_bit_cast(bf16x8, *(const uint4 *)(qrow + 8 * i));

    f32x4 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -__builtin_inff(), l = 0.0f;
    const int32_t ksub = lr >> 2;                 /* 16-token block of the lane's key rows */
    const int32_t *table = c.table + (int64_t)b * c.table_ld;

    for (int32_t it = begin + wave; it < end; it += kAttnWaves) {
        const int32_t t0 = (it < t.sink_chunks ? it : t.first_chunk + it - t.sink_chunks) << 6;
        const int32_t kt = t0 + 16 * ksub, vt = t0 + 16 * q;
        int32_t kid = -1, vid = -1;
        if (kt < t.s.len) kid = table[kt >> c.page_log2];
        if (vt < t.s.len) vid = table[vt >> c.page_log2];
        const bool kok = kid >= 0 && kid < c.pages, vok = vid >= 0 && vid < c.pages;
        uint4 kr[4][DL], vr[DT];
        float ks = 1.0f, vs = 1.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < DL; ++y) kr[x][y] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int x = 0; x < DT; ++x) vr[x] = make_uint4(0, 0, 0, 0);
        if (kok) {
            const int64_t block = (int64_t)kid * c.H + h;
            const uint8_t *at = c.k + (block * c.page + (kt & (c.page - 1)) + (lr & 3)) * D + q * (D / 4);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < DL; ++y) kr[x][y] = *(const uint4 *)(at + 4 * x * D + 16 * y);
            ks = __builtin_bit_cast(float, (uint32_t)c.k_scale[block] << 23);
        }
        if (vok) {
            const int64_t block = (int64_t)vid * c.H + h;
            const uint8_t *at = c.v + (block * D + lr) * c.page + (vt & (c.page - 1));
#pragma unroll
            for (int x = 0; x < DT; ++x) vr[x] = *(const uint4 *)(at + 16 * x * c.page);
            vs = __builtin_bit_cast(float, (uint32_t)c.v_scale[block] << 23);
        }

        f32x4 s[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            s[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int y = 0; y < DL; ++y) {
                s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(kr[x][y].x, kr[x][y].y, ks), qf[2 * y], s[x], 0, 0, 0);
                s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(kr[x][y].z, kr[x][y].w, ks), qf[2 * y + 1], s[x], 0, 0, 0);
            }
        }

        /* every row sees every token of the chunk, or masks */
        const bool inside = t0 + 63 <= t.pos_lo && (!p.window || t0 > t.pos_hi - p.window || t0 + 63 < p.sinks);
        if (!inside || __ballot(!vok) != 0) {
            uint32_t any[4] = {0, 0, 0, 0};       /* bytes of tokens that some row sees */
            uint32_t mine = 0;                    /* tokens that this row sees          */
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const int32_t tk = vt + x;
                if (vok && tk <= pos && (!p.window || tk > pos - p.window || tk < p.sinks)) mine |= 1u << x;
                if (vok && tk <= t.pos_hi && (!p.window || tk > t.pos_lo - p.window || tk < p.sinks)) any[x >> 2] |= 0xFFu << (8 * (x & 3));
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) s[x >> 2][x & 3] = mine >> x & 1u ? s[x >> 2][x & 3] : -__builtin_inff();
            /* tokens that no row sees may hold anything, a NaN too, which
             * a weight of zero would not keep out of the sums */
            uint32_t nan[4] = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < DT; ++x) {
                vr[x] = make_uint4(vr[x].x & any[0], vr[x].y & any[1], vr[x].z & any[2], vr[x].w & any[3]);
                nan[0] |= (vr[x].x & 0x7F7F7F7Fu) + 0x01010101u;
                nan[1] |= (vr[x].y & 0x7F7F7F7Fu) + 0x01010101u;
                nan[2] |= (vr[x].z & 0x7F7F7F7Fu) + 0x01010101u;
                nan[3] |= (vr[x].w & 0x7F7F7F7Fu) + 0x01010101u;
            }
            const uint32_t some = (nan[0] | nan[1] | nan[2] | nan[3]) & 0x80808080u;
            if (__ballot(some != 0) != 0) {
                /* a NaN that some of the rows see: out of the values, and
                 * into the scores of those rows */
                uint32_t tok = 0;
#pragma unroll
                for (int x = 0; x < 16; ++x) tok |= (nan[x >> 2] >> (8 * (x & 3) + 7) & 1u) << x;
                for (int off = 1; off < 16; off <<= 1) tok |= __shfl_xor(tok, off, 64);
                uint32_t clean[4] = {0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    if (tok >> x & 1u) {
                        if (mine >> x & 1u) s[x >> 2][x & 3] = __builtin_nanf("");
                    } else {
                        clean[x >> 2] |= 0xFFu << (8 * (x & 3));
                    }
                }
#pragma unroll
                for (int x = 0; x < DT; ++x)
                    vr[x] = make_uint4(vr[x].x & clean[0], vr[x].y & clean[1], vr[x].z & clean[2], vr[x].w & clean[3]);
            }
        }

        float top = -__builtin_inff();
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3])));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float now = fmaxf(m, top * p.scale_log2);
        const float ref = now == -__builtin_inff() ? 0.0f : now;   /* no token seen yet */
        const float fade = __builtin_amdgcn_exp2f(m - ref);
        m = now;
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][y], p.scale_log2, -ref));
                s[x][y] = e;
                sum += e;
            }
        l = l * fade + sum;
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y] *= fade;
        /* weights enter the second product in 16 bits: each is off by up to
         * 2^-8 of itself, independently, and the output is rounded as far */
        bf16x8 pf[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            pf[x] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16(s[2 * x][0], s[2 * x][1]), pack_bf16(s[2 * x][2], s[2 * x][3]),
                                                          pack_bf16(s[2 * x + 1][0], s[2 * x + 1][1]),
                                                          pack_bf16(s[2 * x + 1][2], s[2 * x + 1][3])));
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            o[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(vr[x].x, vr[x].y, vs), pf[0], o[x], 0, 0, 0);
            o[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(vr[x].z, vr[x].w, vs), pf[1], o[x], 0, 0, 0);
        }
    }

    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    /* join the wavefronts */
    __shared__ float st[kAttnWaves][2][16];
    __shared__ f32x4 red[kAttnWaves][DT][64];
    if (q == 0) {
        st[wave][0][lr] = m;
        st[wave][1][lr] = l;
    }
    __syncthreads();
    float all = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) all = fmaxf(all, st[w][0][lr]);
    const float ref = all == -__builtin_inff() ? 0.0f : all;
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) total += st[w][1][lr] * __builtin_amdgcn_exp2f(st[w][0][lr] - ref);
    const float f = __builtin_amdgcn_exp2f(m - ref);
#pragma unroll
    for (int x = 0; x < DT; ++x) {
        f32x4 v = o[x];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] *= f;
        red[wave][x][lane] = v;
    }
    __syncthreads();
    const int64_t slot = ((int64_t)blockIdx.z * p.row_tiles + blockIdx.y) * p.splits + blockIdx.x;
    for (int32_t x = wave; x < DT; x += kAttnWaves) {
        f32x4 v = red[0][x][lane];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) v += red[w][x][lane];
        if (t.parts > 1)
            *(f32x4 *)(p.part + (slot * DT + x) * 256 + lane * 4) = v;
        else if (r0 + lr < t.rows)
            write_out<D>(p, t, h, r0 + lr, x, q, v, all, total);
    }
    if (t.parts > 1 && threadIdx.x < 16) {
        p.stat[slot * 32 + lr] = all;
        p.stat[slot * 32 + 16 + lr] = total;
    }
}

/* Parts in ascending order; a wavefront takes 16 channels of the 16 rows. */
template <int D>
__global__ __launch_bounds__(D * 4) void attention_combine_kernel(AttnParams p)
{
    constexpr int DT = D / 16;
    const int32_t lane = threadIdx.x & 63, x = threadIdx.x >> 6, lr = lane & 15, q = lane >> 4;
    const int32_t b = blockIdx.y / p.c.H, h = blockIdx.y % p.c.H, r0 = blockIdx.x * 16;
    const Tile t = row_tile(p, b, r0);
    if (r0 + lr >= t.rows || t.parts == 1) return;
    const int64_t slot = ((int64_t)blockIdx.y * p.row_tiles + blockIdx.x) * p.splits;
    float all = -__builtin_inff();
    for (int32_t i = 0; i < t.parts; ++i) all = fmaxf(all, p.stat[(slot + i) * 32 + lr]);
    const float ref = all == -__builtin_inff() ? 0.0f : all;
    float total = 0.0f;
    f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t i = 0; i < t.parts; ++i) {
        const float f = __builtin_amdgcn_exp2f(p.stat[(slot + i) * 32 + lr] - ref);
        total += f * p.stat[(slot + i) * 32 + 16 + lr];
        const f32x4 v = *(const f32x4 *)(p.part + ((slot + i) * DT + x) * 256 + lane * 4);
#pragma unroll
        for (int y = 0; y < 4; ++y) sum[y] += f * v[y];
    }
    write_out<D>(p, t, h, r0 + lr, x, q, sum, all, total);
}

namespace {

template <int D>
hipError_t launch_dim(const AttnParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL(attention_kernel<D>, dim3((uint32_t)p.splits, (uint32_t)p.row_tiles, (uint32_t)(p.c.B * p.c.H)),
                       dim3(kAttnWaves * 64), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL(attention_combine_kernel<D>, dim3((uint32_t)p.row_tiles, (uint32_t)(p.c.B * p.c.H)), dim3(D * 4), 0, stream, p);
    return hipGetLastError();
}

} /* namespace */

hipError_t launch_attention(const AttnParams &p, hipStream_t stream)
{
    if (p.D == 64) return launch_dim<64>(p, stream);
    if (p.D == 128) return launch_dim<128>(p, stream);
    return launch_dim<256>(p, stream);
}

} /* namespace g355 */
