/*
 * serve.h -- launch interface of the serving operators: products with 4-bit
 * weights (w4.hip) and the paged 8-bit key/value cache with the attention that
 * reads it (kvcache.hip).  Internal; not part of the C ABI.
 */
#ifndef GEMM355_SERVE_H
#define GEMM355_SERVE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace g355 {

/* Division of numbers under 2^31 by d: with l = ceil(log2 d) and
 * m = ceil(2^(31 + l) / d), floor(n / d) = floor(n m / 2^(31 + l)), as m exceeds
 * the exact quotient by less than 1 <= 2^l / d. */
struct Divider {
    uint32_t magic;               /* m; 0: d = 1                             */
    int32_t shift;                /* l - 1                                   */
};

inline Divider divider(int64_t d)
{
    int32_t l = 0;
    while (((int64_t)1 << l) < d) ++l;
    return Divider{d == 1 ? 0u : (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d), l - 1};
}

__device__ __forceinline__ int32_t quotient(int32_t n, const Divider &d)
{
    return d.magic ? (int32_t)(__umulhi((uint32_t)n, d.magic) >> d.shift) : n;
}

/* A packed N x K matrix: two codes a byte, element 2i in the low nibble. */
struct W4Params {
    uint8_t *codes;
    int64_t ldb;                  /* bytes between rows, multiple of 16      */
    void *scales;                 /* [N][ng] bf16 (INT) or E8M0 (MXFP4)      */
    uint8_t *zeros;               /* [N][ng] or null                         */
    int32_t N, K, ng;
    int32_t group;                /* 32, 64 or 128                           */
    int32_t mx;                   /* 1: E2M1 codes, E8M0 scales              */
};

struct W4QuantParams {
    W4Params w;
    const void *x;                /* quantise: source; dequantise: unused    */
    void *y;                      /* dequantise: destination                 */
    int64_t ld;                   /* elements between rows of x or y         */
    int32_t f32;                  /* x or y: 1 fp32, 0 bf16                  */
    int32_t vec;                  /* rows of x or y 16-byte aligned          */
    /* set by the launch: octets of a row, the rows of one blockIdx.y */
    int32_t per_row, rows_y;
    Divider by_row;
};

struct W4GemmParams {
    W4Params w;
    const uint16_t *x;            /* bf16 [M][K]                             */
    void *y;                      /* [M][N]                                  */
    int64_t ldx, ldy;             /* elements                                */
    int32_t M;
    int32_t out_bf16;
    int32_t even;                 /* 1: K a multiple of 128, rows of x 16-byte
                                     aligned, scales and zero points aligned
                                     and filling whole dwords              */
    int32_t tiny;                 /* 1: K < 8, or scales or zero points of
                                     less than a dword                      */
    uint32_t spread;              /* set by the launch: 2^32 / workgroups    */
};

hipError_t launch_w4_quantize(const W4QuantParams &p, hipStream_t stream);
hipError_t launch_w4_dequantize(const W4QuantParams &p, hipStream_t stream);
hipError_t launch_w4_gemm(const W4GemmParams &p, hipStream_t stream);

/* A paged cache and the step that runs on it (gemm355_kv_cache). */
struct KvParams {
    uint8_t *k, *v;               /* [pages][H][page][D], [pages][H][D][page] */
    uint8_t *k_scale, *v_scale;   /* [pages][H]                              */
    const int32_t *table;         /* [B][table_ld]                           */
    const int32_t *lens;          /* [B]                                     */
    const int32_t *q_start;       /* [B + 1] or null                         */
    int64_t pages, table_ld;
    int32_t H, page, page_log2;
    int32_t B, tokens, max_new, max_len;
};

struct KvAppendParams {
    KvParams c;
    const uint16_t *xk, *xv, *q;
    uint16_t *q_out;
    int64_t ldk, ldv, ldq, ldqo;  /* elements between tokens                 */
    const float *cos, *sin;       /* [positions][rot / 2] or null            */
    int32_t Hq, D, rot, interleaved;
    int32_t whole;                /* 1: rot a multiple of 16, tables 16-byte
                                     aligned                                */
};

struct AttnParams {
    KvParams c;
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    int64_t ldq, ldo;             /* elements between tokens                 */
    float scale_log2;             /* softmax scale times log2(e)             */
    int32_t Hq, group, D;
    Divider by_group;
    int32_t window, sinks;        /* window 0: none                          */
    int32_t tile_rows;            /* rows a workgroup: 16 or 32              */
    int32_t row_tiles;            /* of max_new * group rows                 */
    int32_t waves;                /* wavefronts a workgroup: of 16 rows 8 (D
                                     64, 128), 4 (D 128, 256) or 2 (D 256);
                                     of 32 rows 4 (D 64, 128) or 2          */
    int32_t splits;               /* parts of the key axis                   */
    int32_t part_chunks;          /* least 64-token chunks a part            */
    float *part;                  /* [B H row_tiles][splits][tile_rows][D]   */
    float *stat;                  /* sums, and their maxima and totals       */
};

hipError_t launch_kv_append(const KvAppendParams &p, hipStream_t stream);
hipError_t launch_attention(const AttnParams &p, hipStream_t stream);

} /* namespace g355 */

#endif
