/*
 * cgdr_serve.h -- the operators of libcgdr that a decoder built on the delta rule needs next to
 * it: the short causal convolution in front of the recurrent layers, the selective state space
 * scan, and, for its full-attention layers, a paged key-value cache held in 8 bits with the
 * block tables, the append and the attention that go with it.  None of them has a counterpart
 * in the pages that cgdr.h cites.
 *
 * Conventions, as in cgdr.h: device pointers, strides in ELEMENTS, innermost dimension
 * contiguous, asynchronous on `stream`, launched on the calling thread's current device, every
 * buffer owned by the caller, nothing allocated, arguments checked on the host before any
 * launch, no C++ exception across the ABI.  No input may alias an output other than the state,
 * cache and table buffers that are named as updated in place.
 *
 * Rows that are read or written as vectors (x, dt, z, B, C, q, k, v, o, and the conv state) need
 * 16-byte aligned base pointers and strides of a multiple of 16 bytes.
 *
 * Packed sequences: with `cu` given (int32 [B+1] on the device, cu[0] = 0, ascending), the rows
 * of sequence b are the packed tokens cu[b] .. cu[b+1]-1 of n_tokens in all, `T` and the batch
 * strides are ignored, and a sequence may be empty (its state then stays).  Offsets outside
 * [0, n_tokens] are clamped: they never make a call read or write outside its tensors.  Without
 * `cu` the rows are [B, T, ...].
 *
 * status words: as in cgdr_args, optional, never cleared by the library.
 */
#ifndef CGDR_SERVE_H_
#define CGDR_SERVE_H_

#include "cgdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Short causal convolution along the tokens, one filter per channel:
 *     y[t, c] = act(bias[c] + sum_{j < W} weight[c, j] * u[t - (W-1) + j, c])
 * where u is the sequence x with the W-1 rows of `state` in front of it, and act is
 * x / (1 + e^-x) (SiLU) or nothing.  Afterwards `state` holds the last W-1 rows of u, so a prompt
 * and the tokens that follow it, in any split, give the rows of one long call.  Sums in fp32.
 */
typedef struct cgdr_conv_args {
    int32_t B, T, C, W;             /* W in 2..4; C a multiple of 8 (bf16) or 4 (fp32) */
    int32_t dtype;                  /* cgdr_dtype of x, o and state */
    int32_t silu;                   /* nonzero: SiLU, else no activation */
    int32_t n_tokens;               /* packed form: rows of x and o */
    int32_t reserved;
    const void *x;  int64_t x_sb, x_st;     /* [B,T,C], or [n_tokens,C] with row stride x_st */
    void *o;        int64_t o_sb, o_st;
    const float *weight;                    /* [C,W] fp32, dense, 16-byte aligned */
    const float *bias;                      /* [C] fp32 or NULL */
    void *state;                            /* [B,W-1,C] dense, oldest row first; in place */
    const int32_t *cu;                      /* [B+1] or NULL */
    int32_t *status;                        /* reserved for the index-checking build */
} cgdr_conv_args;

cgdr_status cgdr_conv(const cgdr_conv_args *args, void *stream);

/*
 * Selective state space scan.  Per channel c (of group g = c / (C/G)) an fp32 state h of N values:
 *     d    = dt[t, c] + dt_bias[c];  d = softplus(d) if `softplus` (softplus(x) = x for x > 20)
 *     h[n] = exp(-exp(A_log[c, n]) d) h[n] + d x[t, c] B[t, g, n]
 *     y    = sum_n C[t, g, n] h[n] + D[c] x[t, c]
 *     o    = y, or y z / (1 + e^-z) with the gate z
 * T == 1 without `cu` is the single-token form (each state value read and written once).
 * Longer sequences are cut into chunks of tokens when the channels alone leave SMs idle: a first
 * launch forms every chunk's end state, a second runs the chunks from the states joined from
 * these.  `workspace` (16-byte aligned) holds them; cgdr_scan_workspace_size may be 0.
 */
typedef struct cgdr_scan_args {
    int32_t B, T, C, N, G;          /* N in {16, 32, 64, 128}; C/G a multiple of 8; B <= 32768 */
    int32_t dtype;                  /* cgdr_dtype of x, dt, z, B, C */
    int32_t o_dtype;                /* cgdr_dtype of o */
    int32_t softplus;
    int32_t n_tokens;
    int32_t reserved;
    const void *x;  int64_t x_sb, x_st;         /* [B,T,C] */
    const void *dt; int64_t dt_sb, dt_st;       /* [B,T,C] */
    const void *z;  int64_t z_sb, z_st;         /* [B,T,C] or NULL */
    const void *Bm; int64_t Bm_sb, Bm_st;       /* [B,T,G,N], groups dense */
    const void *Cm; int64_t Cm_sb, Cm_st;       /* [B,T,G,N], groups dense */
    void *o;        int64_t o_sb, o_st;         /* [B,T,C] */
    const float *A_log;                         /* [C,N] dense, 16-byte aligned */
    const float *D;                             /* [C] or NULL, 8-byte aligned */
    const float *dt_bias;                       /* [C] or NULL, 8-byte aligned */
    float *state;                               /* [B,C,N] dense; in place */
    const int32_t *cu;                          /* [B+1] or NULL */
    int32_t *status;                            /* reserved for the index-checking build */
} cgdr_scan_args;

size_t cgdr_scan_workspace_size(const cgdr_scan_args *args);
cgdr_status cgdr_scan(const cgdr_scan_args *args, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Block tables and slots of a step, from the requests' lengths, without the host.  Request b holds
 * seq_lens[b] cached tokens in the first ceil(seq_lens[b] / page) entries of its table row, and
 * gets new_lens[b] tokens more.  The pages that this needs are taken off the top of the stack
 * free_pages[0 .. *free_count - 1], in request order, and entered into block_table; then
 *     cu[b]       prefix sum of new_lens ([B+1])
 *     kv_lens[b]  = seq_lens[b] + new_lens[b]
 *     requests[i], positions[i], slots[i]  of packed new token i: its request, its place in the
 *                 request, and page * page_size + place in the page (int64); -1 from the last
 *                 new token to n_tokens
 *     *free_count_out  the pages left.
 * All or nothing: where the free pages, a table row's width or n_tokens do not suffice
 * (CGDR_ERR_CAPACITY in `status`), or a length is negative, a free count outside [0, F] or a taken
 * page outside [0, num_pages) (CGDR_ERR_INVALID_ARG in `status`), the table keeps its entries,
 * kv_lens = seq_lens, *free_count_out = *free_count, cu is all zero and every slot is -1.
 */
typedef struct cgdr_plan_args {
    int32_t B, width, page;         /* B in 0..8192; page in {16, 32, 64, 128} */
    int32_t n_tokens;               /* entries of requests, positions and slots */
    int32_t F;                      /* entries of free_pages */
    int32_t num_pages;              /* pages of the cache */
    int32_t *block_table;           /* [B,width], row stride table_sb; in place */
    int64_t table_sb;
    const int32_t *seq_lens, *new_lens;         /* [B] */
    const int32_t *free_pages, *free_count;     /* [F], [1] */
    int32_t *free_count_out;                    /* [1], another word than free_count */
    int32_t *kv_lens, *cu;                      /* [B], [B+1] */
    int32_t *requests, *positions;              /* [n_tokens] */
    int64_t *slots;                             /* [n_tokens], 8-byte aligned */
    int32_t *status;
} cgdr_plan_args;

cgdr_status cgdr_cache_plan(const cgdr_plan_args *args, void *stream);

/*
 * The 8-bit cache: k_cache and v_cache int8 [num_pages, Hkv, page, D], dense, with one fp32 scale
 * for each (page, head) in k_scale and v_scale [num_pages, Hkv]; a value is scale * int8.
 *
 * Append: packed token i of k and v goes to slots[i] (page * page_size + offset; below 0: nowhere).
 * Tokens that go to one page are consecutive and ascend, as cgdr_cache_plan lays them out.  Per
 * (page, head) the scale becomes max(old, amax * r) over the new values, r = 1/127 rounded to fp32 (one
 * unit in the last place from the quotient at most), with old = 0 where the first new token enters the
 * page at offset 0 (what a page held for an earlier request plays no part); where it grows, the values
 * already in the page are rounded to it.  To nearest, ties to even, of the IEEE quotient by the scale.  A NaN or an infinity makes the scale of its page and head
 * non-finite, and with it every value of that page and head.
 * A slot outside the cache is skipped and reported as CGDR_ERR_BOUNDS.
 */
typedef struct cgdr_append_args {
    int32_t n, Hkv, D, page;        /* D in {32, 64, 128} */
    int32_t dtype;                  /* cgdr_dtype of k and v */
    int32_t num_pages;
    const void *k;  int64_t k_st, k_sh;     /* [n,Hkv,D] */
    const void *v;  int64_t v_st, v_sh;
    const int64_t *slots;                   /* [n] */
    int8_t *k_cache, *v_cache;              /* in place, 16-byte aligned */
    float *k_scale, *v_scale;               /* in place */
    int32_t *status;
} cgdr_append_args;

cgdr_status cgdr_cache_append(const cgdr_append_args *args, void *stream);

/*
 * Attention of the n newest tokens over the cache.  Query token j (of q_len = cu[b+1] - cu[b]) of
 * request b stands at position kv_lens[b] - q_len + j and sees the positions up to its own; query
 * head h reads key-value head h / (Hq/Hkv).  softmax(scale q.k) v, softmax and sums in fp32; a row
 * that sees nothing (kv_lens[b] < q_len) is zero.  `max_q` and `max_kv` bound q_len and kv_lens on
 * the host (they size the launch): what exceeds them, or the table's width * page, is cut off and
 * reported as CGDR_ERR_CAPACITY, rows of o beyond max_q stay as they are.  Table entries past a request's pages are not read; a page
 * outside [0, num_pages) is left out of the sums and reported as CGDR_ERR_BOUNDS.
 * Where rows are few, key-value positions are split over CTAs; `workspace` (16-byte aligned) holds the parts.
 * A wait that gives up reports CGDR_ERR_TIMEOUT in *status; the rows of its CTA are then undefined.
 * bf16: products of fp16 operands (int8 values are exact in fp16, queries are scaled by a power of
 * two per row first).  fp32: both queries and probabilities in two fp16 parts.  A page's v scale below 2^-100 counts as
 * zero; a NaN in a scale reaches the rows that see its page, and no others.
 */
typedef enum cgdr_attend_path {
    CGDR_ATTEND_AUTO = 0,           /* per call: whichever of the two measured less time where every request has max_q
                                       query tokens and max_kv cached ones; a long prompt among many single tokens
                                       over long caches takes less in a call of its own */
    CGDR_ATTEND_ROWS = 1,           /* row tiles of 8 or 16; a CTA a tile, or the cache split evenly over all SMs */
    CGDR_ATTEND_TILES = 2           /* tensor memory, row tiles of 128, the cache in parts where they are few (bf16,
                                       D = 128, o in 16-byte rows; elsewhere ROWS) */
} cgdr_attend_path;

typedef struct cgdr_attend_args {
    int32_t B, n, Hq, Hkv, D, page, width;
    int32_t dtype;                  /* cgdr_dtype of q and o */
    int32_t num_pages;
    int32_t max_q, max_kv;
    int32_t path;                   /* cgdr_attend_path of this call */
    int32_t wait_polls;             /* polls before a device wait of TILES gives up; 0: 2^18; below 0 (tests): -wait_polls,
                                       and the first wait of every CTA is for something that never comes */
    float scale;                    /* <= 0 selects 1/sqrt(D) */
    const void *q;  int64_t q_st, q_sh;     /* [n,Hq,D] */
    void *o;        int64_t o_st, o_sh;
    const int8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *block_table; int64_t table_sb;
    const int32_t *kv_lens, *cu;            /* [B], [B+1] */
    int32_t *status;
} cgdr_attend_args;

size_t cgdr_cache_attend_workspace_size(const cgdr_attend_args *args);
cgdr_status cgdr_cache_attend(const cgdr_attend_args *args, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CGDR_SERVE_H_ */
