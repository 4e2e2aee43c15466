/*
 * cgdr_layer.h -- the operators of libcgdr around a layer's state: the root-mean-square norm that
 * precedes a layer, the 8-bit operands and matrix products of its projections, and the rotary
 * positions of its queries and keys.  None of them has a counterpart in the pages that cgdr.h cites.
 *
 * Conventions, as in cgdr.h and cgdr_serve.h: device pointers, strides in ELEMENTS, innermost
 * dimension contiguous, asynchronous on `stream`, launched on the calling thread's current device,
 * every buffer owned by the caller, nothing allocated, no workspace, arguments checked on the host
 * before any launch, no C++ exception across the ABI.  No input may alias an output other than the
 * buffers that are named as updated in place and the norm's o, which may be x; equal addresses are
 * refused, overlaps of other kinds are not looked for.  Rows need 16-byte aligned base pointers and strides
 * of a multiple of 16 bytes; rows that a call writes may not overlap.
 *
 * 8 bits: e4m3 values (sign, four exponent bits, three of mantissa, no infinity, largest 448) with
 * fp32 scales; a value is scale * e4m3.  Rows have a scale for each 128 consecutive values (the last
 * group may be shorter), weights one for each block of 128 x 128.  Of a group's largest magnitude,
 *     scale = max(amax * r, 2^-126)       r = 1/448 rounded to fp32
 *     e4m3  = x * (1/scale), each step rounded to fp32, then to nearest (ties to even), at most 448
 * so zeros stay zeros, and a NaN or an infinity makes its group's scale non-finite and with it every
 * value of that group, and no other.
 *
 * status words: as in cgdr_args, optional, never cleared by the library.
 */
#ifndef CGDR_LAYER_H_
#define CGDR_LAYER_H_

#include "cgdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm of rows x [n,H,C], with the residual's addition:
 *     h = x + residual;  residual <- h (rounded to its type)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 * h, the mean and y in fp32; y is formed from h as it was before it was rounded.  The output is o, in
 * dtype, or y8 with its scales.  The squares of a row are added up before they are divided by C: a row whose sum(h^2)
 * overflows fp32 (3.4e38: one value above 1.8e19, or C = 4096 values above 2.9e17 each) becomes zero.
 */
typedef struct cgdr_norm_args {
    int32_t n, H, C;                /* C a multiple of 8, at most 32768; H == 1 with y8 */
    int32_t dtype;                  /* cgdr_dtype of x, residual and o */
    float eps;                      /* < 0 selects 1e-6 */
    const void *x;  int64_t x_st, x_sh;         /* [n,H,C] */
    void *residual; int64_t residual_st, residual_sh;         /* [n,H,C] or NULL; in place */
    const float *weight;                        /* [C], 16-byte aligned, or NULL for ones */
    void *o;        int64_t o_st, o_sh;         /* [n,H,C], or NULL with y8; may be x, with its strides */
    void *y8;       int64_t y8_st;              /* [n,C], or NULL with o */
    float *y_scale;                             /* [n, ceil(C/128)] dense */
    int32_t *status;                            /* reserved for the index-checking build */
} cgdr_norm_args;

cgdr_status cgdr_norm(const cgdr_norm_args *args, void *stream);

/*
 * x [n,C] in 8 bits: of rows (block_rows == 1, a scale for each 128 values) or of weights
 * (block_rows == 128, a scale for each block of 128 x 128).
 */
typedef struct cgdr_quantize_args {
    int32_t n, C;                   /* C a multiple of 8 */
    int32_t dtype;                  /* cgdr_dtype of x */
    int32_t block_rows;             /* 1 or 128 */
    const void *x;  int64_t x_st;   /* [n,C] */
    void *y8;       int64_t y8_st;  /* [n,C] */
    float *y_scale;                 /* [ceil(n/block_rows), ceil(C/128)] dense */
    int32_t *status;                /* reserved for the index-checking build */
} cgdr_quantize_args;

cgdr_status cgdr_quantize(const cgdr_quantize_args *args, void *stream);

/*
 * o = x w^T of 8-bit operands, x [n,K] with x_scale [n,KB], w [N,K] with w_scale [NB,KB]; KB and NB
 * are K and N over 128, rounded up:
 *     o[i,j] = sum_b x_scale[i,b] w_scale[j/128,b] sum_{k of block b} x[i,k] w[j,k]
 * Products are exact, sums are fp32; x_scale w_scale is formed first, in fp32, so scales whose product
 * overflows give infinities or NaN.  Rows of x and of w may not overlap (they are described to the copy
 * engine).  A NaN or an infinity reaches the outputs of its row of x, or of its rows of w, and no others.
 * `path` says which kernel runs (they agree up to the order of sums).  A wait that gives
 * up reports CGDR_ERR_TIMEOUT in *status; the outputs of its CTA (or cluster) are then undefined.
 */
typedef enum cgdr_matmul_path {
    CGDR_MATMUL_AUTO = 0,           /* per call: whichever of the two measured less time */
    CGDR_MATMUL_FEW = 1,            /* few rows of x: 128 rows of w a CTA, K in parts over a cluster */
    CGDR_MATMUL_TILES = 2           /* tiles of 128 rows of x by 128 or 256 rows of w */
} cgdr_matmul_path;

typedef struct cgdr_matmul_args {
    int32_t n, N, K;
    int32_t o_dtype;                /* cgdr_dtype of o */
    int32_t path;                   /* cgdr_matmul_path of this call */
    int32_t wait_polls;             /* polls before a device wait gives up; 0: 2^18; below 0 (tests): -wait_polls,
                                       and the first wait of every CTA is for something that never comes */
    const void *x;  int64_t x_st;   /* [n,K] e4m3 */
    const float *x_scale;           /* [n,KB] dense */
    const void *w;  int64_t w_st;   /* [N,K] e4m3 */
    const float *w_scale;           /* [NB,KB] dense */
    void *o;        int64_t o_st;   /* [n,N] */
    int32_t *status;
} cgdr_matmul_args;

cgdr_status cgdr_matmul(const cgdr_matmul_args *args, void *stream);

/*
 * Rotary positions: the first R = 2 * half channels of every head of q [n,Hq,D] and k [n,Hk,D] are turned in
 * pairs, in place.  Pair i of token t turns by a = positions[t] * freq[i]:
 *     (u, v) <- scale * (u cos a - v sin a, v cos a + u sin a)
 * u and v are channels i and i + half, or 2 i and 2 i + 1 (interleaved).  a is formed modulo a turn in 64
 * bits, so positions up to 2^31 lose nothing; cos, sin and the products are fp32.  Of frequencies of 6e-12 and
 * more (2^24 steps of 2^-64 turns) cos and sin are good to fp32's relative rounding, however small they are.  Tokens
 * with a position below 0 stay as they are.
 */
typedef struct cgdr_rotary_args {
    int32_t n, Hq, Hk, D;           /* Hk may be 0 */
    int32_t half;                   /* 2 * half <= D; at most 256 */
    int32_t dtype;                  /* cgdr_dtype of q and k */
    int32_t interleaved;
    float scale;
    void *q;  int64_t q_st, q_sh;   /* [n,Hq,D]; in place */
    void *k;  int64_t k_st, k_sh;   /* [n,Hk,D] or NULL; in place; not q */
    const int32_t *positions;       /* [n] */
    const double *freq;             /* [half], radians a position */
    int32_t *status;                /* reserved for the index-checking build */
} cgdr_rotary_args;

cgdr_status cgdr_rotary(const cgdr_rotary_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CGDR_LAYER_H_ */
