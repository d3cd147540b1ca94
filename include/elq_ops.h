/*
 * elq_ops.h -- C ABI of the 8-bit-integer expert path and the norms around a
 * block, for B200 (sm_100a).  Same library (libelq.so), statuses and
 * conventions as elq.h; this header adds to it and changes none of it.
 *
 * Where the layer of elq.h quantises activations in blocks of 32 (Q8_1) and so
 * rescales every 32 products, the calls here give a whole row of activations
 * one scale and every output channel of a weight matrix one scale: a row dot
 * is one exact int32 sum, rescaled once.  The calls chain to a whole expert
 * block (pre-norm to codes, D product, elq_router_topk, elq_route_bucket,
 * gather and quantise, grouped gate/up, SwiGLU and quantise, grouped down,
 * weighted combine and quantise, U product, post-norm with gate and residual),
 * and each stands by itself.
 *
 * Conventions, in addition to elq.h's
 *  - Matrices are row-major with a leading dimension in elements (ld >= the
 *    row's length; the elements between are neither read as values nor
 *    written).  Base pointers are 16-byte aligned, fp32 vectors (scales, norm
 *    weights, bias) 4-byte aligned.  A leading dimension may be any number
 *    where nothing else is said; rows whose bytes are whole multiples of 16
 *    apart are read and written by wide accesses, others element by element.
 *  - Types: ELQ_F32, ELQ_BF16, ELQ_F16 and, where said, ELQ_I8.
 *  - Sums, norms and softmax weights are fp32, integer sums int32; each output
 *    is rounded once, to nearest even, to its type.
 *  - Rows, channels and columns number at most 2^30 each.
 *  - No workspace, no allocation, nothing kept between calls but what elq.h
 *    names; any stream, capturable; calls share nothing on the GPU but the error
 *    word below.  One kernel a call.
 *    An output may not overlap an input, except where in-place use is said.
 *  - Every sum runs in a fixed order: the same call gives the same bits.
 *  - Device data out of range (row indices, positions, group offsets) never
 *    makes an access out of bounds; what it gives instead is said per call.
 *
 * 8-bit rows: a row x of K values becomes codes q (int8, -127 .. 127) and one
 * fp32 scale s = amax / 127 (amax = max |x|, one correctly rounded division);
 * q is x / s rounded to the nearest whole number, halves away from zero -- the
 * exact quotient's, not a rounded quotient's -- and clamped to +-127 (which
 * happens only where s is subnormal).  An all-zero row has s = 0 and zero codes.
 * A row that holds an infinity or a NaN has s = NaN and zero codes, so that a
 * product with it is NaN and the other rows are untouched.
 */
#ifndef ELQ_OPS_H
#define ELQ_OPS_H

#include "elq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {                          /* more GGUF type ids */
    ELQ_F16 = 1,
    ELQ_I8 = 24
};

/* ---- activation rows to codes ------------------------------------------------ */

/* Row quantiser, optionally of gathered rows: output row i is source row
 * index[i] / div (index: device int32 [rows]; e.g. the pair order perm of
 * elq_route_bucket with div = k), or source row i where index is NULL (then
 * div is 1 and rows <= x_rows).  An index that is negative or names a row past
 * x_rows (>= 1) gives a zero row.  x: device [x_rows][cols], x_type F32, BF16 or F16,
 * leading dimension ldx.  q: device int8 [rows][cols], ldq a multiple of 16;
 * scale: device fp32 [rows].  Also gives a weight matrix [N][K] its codes and
 * per-channel scales. */
elq_status elq_quantize_i8(const void* x, int32_t x_type, int64_t x_rows, int32_t cols, int64_t ldx,
                           const int32_t* index, int32_t div, int64_t rows, int8_t* q, int64_t ldq,
                           float* scale, void* stream);

/* SwiGLU, then the row quantiser: row i of gu is I gate values, then I up
 * values (ld >= 2 I); h = (g / (1 + exp(-g))) * u in fp32, within 5 * 2^-24 of its
 * value (or 2^-119 |u| where g < -87, or 2^-149), quantised to q [rows][I] and scale
 * [rows]. */
elq_status elq_swiglu_i8(const void* gu, int32_t x_type, int64_t rows, int32_t I, int64_t ld, int8_t* q,
                         int64_t ldq, float* scale, void* stream);

/* Weighted combine, then the row quantiser: y[t] = sum over j < k, in order,
 * of weights[t][j] * o[pos[t][j]] in fp32 (fused multiply-adds from 0),
 * quantised to q [T][cols] and scale [T].  o: device [o_rows][cols], o_type F32,
 * BF16 or F16; pos: device int32 [T][k] (elq_route_bucket's); weights: device
 * fp32 [T][k]; k <= 64.  A position outside 0 .. o_rows-1 adds nothing (o_rows >= 1). */
elq_status elq_combine_i8(const void* o, int32_t o_type, int64_t o_rows, int32_t cols, int64_t ldo,
                          const int32_t* pos, const float* weights, int64_t T, int32_t k, int8_t* q,
                          int64_t ldq, float* scale, void* stream);

/* ---- products -------------------------------------------------------------------- */

/* y[t][n] = (sum_k x[t][k] * w[n][k]) * sx[t] * sw[n] (+ bias[n]): 8-bit codes,
 * an exact int32 sum, one scale a token and one a channel (in this order, each
 * operation one fp32 rounding, so that all forms of it agree).  x: device int8
 * [T][K]; sx: device fp32 [T]; w: device int8 [N][K]; sw: device fp32 [N];
 * bias: device fp32 [N] or NULL; y: device [T][N], y_type F32, BF16 or F16.
 * ldx and ldw multiples of 16; 1 <= K <= 65536, N >= 1. */
elq_status elq_i8_matmul(const int8_t* x, int64_t ldx, const float* sx, int64_t T, const int8_t* w, int64_t ldw,
                         const float* sw, const float* bias, int32_t N, int32_t K, void* y, int32_t y_type,
                         int64_t ldy, void* stream);

/* Products grouped by expert: rows offsets[e] .. offsets[e+1]-1 of x times
 * expert e's matrix, y[r][n] = sum_k x[r][k] * w[e][n][k] (times sx[r] * sw[e][n]
 * for codes).  x: device [M][K]; w: device [E][N][K], ldw between rows, w_stride
 * (elements, >= (N-1) * ldw + K) between experts; both x_type: I8 (with sx [M]
 * and sw [E][N]), BF16 or F16 (sx and sw NULL; fp32 accumulation).  y: device
 * [M][N], y_type F32 or, for I8, BF16 or F16; for 16-bit x F32 or x_type.
 * offsets: device int32 [E+1], non-decreasing, as elq_route_bucket writes them
 * (each is taken as clamped to 0 .. M and raised to the largest before it, so
 * that groups are disjoint whatever the array holds).  Rows outside every group
 * are left as they were.  Rows of x and w and experts of w are whole multiples of
 * 16 bytes apart (ldx, ldw, w_stride); 1 <= K <= 65536, 1 <= E <= 1024. */
elq_status elq_grouped_matmul(const void* x, int32_t x_type, int64_t ldx, const float* sx, int64_t M, const void* w,
                              int64_t ldw, int64_t w_stride, const float* sw, int32_t E, int32_t N, int32_t K,
                              const int32_t* offsets, void* y, int32_t y_type, int64_t ldy, void* stream);

/* ---- norms around a block ------------------------------------------------------- */

/* The norm before a block: n[t] = x[t] / sqrt(mean(x[t]^2) + eps) * weight.
 * x: device [T][cols], x_type F32, BF16 or F16; weight: device fp32 [cols] or
 * NULL (ones); eps > 0.  n: device [T][cols], n_type F32, BF16, F16, or I8: the
 * fp32 norm handed straight to the row quantiser (ldn a multiple of 16, scale:
 * device fp32 [T]; else scale is NULL).  n may be x itself where their types
 * and leading dimensions agree.  |x| up to 1e36. */
elq_status elq_rms_norm(const void* x, int32_t x_type, int64_t T, int32_t cols, int64_t ldx, const float* weight,
                        float eps, void* n, int32_t n_type, int64_t ldn, float* scale, void* stream);

/* The norm after a block, with its gate and residual, and the next block's
 * norm, in one pass:
 *   v  = y[t] / sqrt(mean(y[t]^2) + eps) * post_weight
 *   h' = res_scale * h[t] + gate * v
 *   n  = h' / sqrt(mean(h'^2) + eps) * next_weight        (of the unrounded h')
 * All of it fp32 (where all rows share the gate it meets post_weight first), h'
 * and n each rounded once; |y| and |h'| up to 1e36. */
typedef struct {
    int64_t T;
    int32_t cols;
    int32_t h_type, y_type, n_type;     /* h, h_out: F32, BF16, F16; y: likewise; n: those or I8 */
    const void* h;                      /* device [T][cols] */
    const void* y;                      /* device [T][cols] */
    const float* post_weight;           /* device fp32 [cols], or NULL: ones */
    const float* gate;                  /* device fp32 [ceil(T / gate_rows)][gate_cols], or NULL: ones */
    const float* next_weight;           /* device fp32 [cols], or NULL: ones */
    void* h_out;                        /* device [T][cols] of h_type; may be h itself (ld_out = ldh) */
    void* n;                            /* device [T][cols] of n_type, or NULL: no next norm */
    float* scale;                       /* device fp32 [T] for n_type I8, else NULL */
    int64_t ldh, ldy, ld_out, ldn;      /* ldn a multiple of 16 for I8 */
    int64_t gate_rows;                  /* >= 1: row t takes gate row t / gate_rows (T or more: one row for all) */
    int64_t gate_ld;                    /* between gate rows */
    int32_t gate_cols;                  /* cols: one value a channel; 1: one value a row */
    float res_scale, eps;               /* eps > 0 */
} elq_residual;

elq_status elq_residual_norm(const elq_residual* r, void* stream);

/* ---- status ---------------------------------------------------------------------- */

/* Blocking: synchronises `stream` (and no other), reads the current device's error
 * word of the calls in this header and clears it, in one step; ELQ_OK, or
 * ELQ_ERR_TIMEOUT if a bounded device wait of a product ran out since the last read
 * (its y is undefined). */
elq_status elq_ops_status(void* stream);

/* ---- test entry point --------------------------------------------------------------- */

/* Failure detection of the products: elq_i8_matmul on the tensor cores with a wait
 * that cannot end.  stall 1: the copies of the first tile stop one K step short; 2: no
 * accumulator is given back, so that a CTA's (or a pair's) third tile waits for good
 * (a product that gives none a third tile is not disturbed).  The wait runs out after
 * budget_ns (1 ms .. 2 s); the kernel lets its copies and MMAs in flight end and
 * returns, and elq_ops_status then says ELQ_ERR_TIMEOUT.  y is left undefined.
 * ELQ_ERR_UNSUPPORTED where the product does not take the tensor cores. */
elq_status elq_test_i8_matmul_timeout(const int8_t* x, int64_t ldx, const float* sx, int64_t T, const int8_t* w,
                                      int64_t ldw, const float* sw, int32_t N, int32_t K, float* y, int64_t ldy,
                                      int32_t stall, uint64_t budget_ns, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ELQ_OPS_H */
