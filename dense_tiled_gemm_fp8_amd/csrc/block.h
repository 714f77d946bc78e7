/*
 * block.h -- launch interface of the block-scaled operators: the quantiser and
 * the norm (norm.hip), the product and the gated pair of products (block.hip).
 * Internal; not part of the C ABI.
 */
#ifndef GEMM355_BLOCK_H
#define GEMM355_BLOCK_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace g355 {

/* E4M3 codes with an fp32 scale for each block of 128 K-values: of one row
 * (scales [K blocks][lds]), or of 128 rows (scales [row blocks][lds]). */
struct BlockMat {
    uint8_t *codes;
    float *scales;
    int64_t ld;                   /* bytes between rows                      */
    int64_t lds;                  /* floats between K blocks or row blocks   */
};

struct BlockQuantParams {
    BlockMat q;
    const void *x;
    int64_t ldx;                  /* elements                                */
    int32_t rows, K;
    int32_t f32;                  /* x: 1 fp32, 0 bf16                       */
    int32_t block_rows;           /* 1 or 128                                */
};

struct NormParams {
    const void *x, *residual, *weight;
    void *sum, *y;                /* sum null: not stored; y null: codes only */
    BlockMat q;                   /* codes null: none                        */
    int64_t ldx, ldr, lds, ldy;   /* elements                                */
    int32_t rows, width;
    int32_t x_f32, r_f32, w_f32, y_f32;
    float eps;
};

/* Products of x (rows of their own scale) with one matrix or two. */
struct BlockGemmParams {
    const uint8_t *x, *w, *up;
    const float *xs, *ws, *us;
    int64_t ldx, ldw, ldu;        /* bytes                                   */
    int64_t lxs, lws, lus;        /* floats                                  */
    int32_t M, N, K, nk;          /* nk: K blocks                            */
    int32_t two;                  /* 1: w and up, 0: w alone                 */
    int32_t act;                  /* of two: 0 SiLU, 1 GELU (tanh)           */
    void *y;                      /* rows, or null: codes                    */
    int64_t ldy;
    int32_t y_f32;
    BlockMat q;
    /* the plan (block_plan) */
    int32_t exact;                /* 1: products exact, every sum of 32 bits */
    int32_t form;                 /* kernel: index of its table              */
    int32_t resident;             /* workgroups that run at once             */
    int32_t splits;               /* parts of K; more than one, or rows that
                                     wait for their scale, go through `part` */
    int32_t part_planes;          /* 0: none; fp32 planes [M][ldp] a part    */
    int64_t ldp;
    float *part;
};

/* Fills the plan for `cus` compute units (splits > 0: that many parts, as far as
 * there are K blocks); the most workgroups of its launches. */
int64_t block_plan(BlockGemmParams &p, int32_t splits, int32_t cus);

hipError_t launch_block_quantize(const BlockQuantParams &p, hipStream_t stream);
hipError_t launch_rmsnorm(const NormParams &p, hipStream_t stream);
hipError_t launch_block_gemm(const BlockGemmParams &p, hipStream_t stream);

} /* namespace g355 */

#endif
