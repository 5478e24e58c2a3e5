/*
 * htroute.h -- C ABI of the expert routing that stands before a grouped product: which rows go to
 * which expert, in the order and with the offsets that gemm_run_grouped, gemm_scaled_run and
 * gemm_int8_run take, the rows themselves from the tokens and back, weighted, with the gradients of
 * both ways, and the loss that keeps the experts evenly used, with its gradient.
 *
 * Status codes and element types are those of htgemm.h.  The caller owns every device buffer and
 * the stream; calls are asynchronous; the buffers and the stream belong to the current device.
 * Results do not depend on scheduling: counts are integers, sums are taken in a fixed order.
 */
#ifndef HTROUTE_H
#define HTROUTE_H

#include "htgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROUTE_MAX_EXPERTS 1024
#define ROUTE_MAX_TOPK 64

/* Device workspace that route_experts and balance_loss need for these sizes (either may use the
 * same one in turn on one stream); 16-byte aligned.  Never 0. */
int route_workspace_size(int64_t tokens, int32_t topk, int32_t experts, size_t* bytes);

/* Assignment t * topk + j sends token t to expert ids[t * ld_ids + j].  It is dropped when that id
 * is outside [0, experts) or mask[t] is 0.
 *   counts[e]   the assignments of expert e
 *   offsets[e]  where e's rows start: offsets[0] = 0, offsets[e+1] = offsets[e] + counts[e] rounded
 *               up to `align`
 *   order[p]    the assignment at row p, in order of the assignments within each expert, -1 in rows
 *               that hold none (the fill up to `align`, and all rows from offsets[experts] on)
 *   slot[t * topk + j]  the row of the assignment, -1 when it is dropped */
typedef struct route_args {
  const int32_t* ids;
  const uint8_t* mask;        /* NULL: every token counts                                           */
  int64_t tokens, ld_ids;
  int32_t topk;               /* 1..ROUTE_MAX_TOPK                                                  */
  int32_t experts;            /* 1..ROUTE_MAX_EXPERTS                                               */
  int32_t align;              /* 1..1024                                                            */
  int32_t* counts;            /* experts values                                                     */
  int32_t* offsets;           /* experts + 1 values                                                 */
  int32_t* order;             /* `rows` values, or NULL                                             */
  int64_t rows;               /* at least tokens * topk + experts * (align - 1) when order is given */
  int32_t* slot;              /* tokens * topk values, or NULL                                      */
  void* workspace;
} route_args;
int route_experts(const route_args* args, void* stream);

/* The balance loss of router logits x (tokens x experts) and the counts of route_experts:
 *
 *   p = softmax(x) by rows;  prob[e] = mean of p(t, e) over the n tokens with mask[t] != 0;
 *   loss = coef * sum over e of (experts * counts[e] / (topk * n)) * prob[e]
 *
 * which is coef when all is even.  p is fp32; the sums over tokens are double, but for the up to four
 * rows that are added at once and one rounding to fp32 of each wave's and workgroup's sum.  A row whose
 * logits are all -infinity has p = 0; a NaN or a +infinity in a row that counts makes the loss NaN;
 * masked rows are not looked at.  With n == 0 loss and prob are 0.  live receives n. */
typedef struct balance_args {
  const void* logits;
  int32_t type;               /* GEMM_F32, GEMM_F16 or GEMM_BF16                                    */
  int32_t experts, topk;
  float coef;
  int64_t tokens, ld;         /* row stride of logits, >= experts                                   */
  const uint8_t* mask;        /* NULL: every token counts                                           */
  const int32_t* counts;
  float* loss;                /* 1 value                                                            */
  float* prob;                /* experts values                                                     */
  int32_t* live;              /* 1 value                                                            */
  void* workspace;
} balance_args;
int balance_loss(const balance_args* args, void* stream);

/* Its gradient with respect to the logits, the counts being constants:
 *
 *   d_logits(t, e) = p(t, e) * (g(e) - sum over f of p(t, f) g(f)),
 *   g(e) = d_loss * coef * experts * counts[e] / (topk * n * n)
 *
 * and 0 in masked rows (every row is written).  live is what balance_loss wrote; d_loss is one
 * device value.  d_logits has the type of logits and row stride ld_d. */
typedef struct balance_grad_args {
  const void* logits;
  int32_t type, experts, topk;
  float coef;
  int64_t tokens, ld;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* live;
  const float* d_loss;
  void* d_logits;
  int64_t ld_d;
} balance_grad_args;
int balance_grad(const balance_grad_args* args, void* stream);

/* ---- tokens to their experts' rows and back --------------------------------------------------- */
/* Up to 2^23 tokens, 2^26 rows and 2^24 columns. */

/* The rows of a routing from the tokens, by order and slot of route_experts:
 *
 *   y(p, :) = x(order[p] / topk, :),  zeros where order[p] is outside [0, tokens * topk)
 *
 * Every one of the `rows` rows is written; y may not overlap x.  The result goes by order alone; slot
 * lets a token be read once for all its rows, and may be NULL.  Its gradient is route_combine without
 * weights. */
typedef struct gather_args {
  const void* x;              /* tokens x cols, row stride ldx                                      */
  int32_t type;               /* GEMM_F32, GEMM_F16 or GEMM_BF16, of x and y                        */
  int32_t topk;               /* 1..ROUTE_MAX_TOPK                                                  */
  int64_t tokens, cols, ldx;
  const int32_t* order;       /* `rows` values                                                      */
  const int32_t* slot;        /* tokens * topk values, or NULL                                      */
  void* y;                    /* rows x cols, row stride ldy                                        */
  int64_t rows, ldy;
} gather_args;
int route_gather(const gather_args* args, void* stream);

/* The tokens from the rows of a routing:
 *
 *   out(t, :) = add(t, :) + sum over j of weights[t * topk + j] * y(slot[t * topk + j], :)
 *
 * in fp32, the terms one after the other, rounded once.  Assignments whose slot is outside [0, rows)
 * add nothing (their weight and no row is looked at); without weights every weight is 1, without add
 * the sum starts from 0.  out may be add, with the same stride; it may not overlap y. */
typedef struct combine_args {
  const void* y;              /* rows x cols, row stride ldy                                        */
  int32_t type;               /* of y, add and out                                                  */
  int32_t weight_type;        /* GEMM_F32, GEMM_F16 or GEMM_BF16; any of them without weights       */
  int64_t rows, cols, ldy;
  const int32_t* slot;        /* tokens * topk values                                               */
  const void* weights;        /* tokens * topk values, or NULL                                      */
  const void* add;            /* tokens x cols, row stride ld_add, or NULL                          */
  int64_t ld_add;
  void* out;                  /* tokens x cols, row stride ld_out                                   */
  int64_t ld_out, tokens;
  int32_t topk;
} combine_args;
int route_combine(const combine_args* args, void* stream);

/* Its gradients, from d_out (that of add is d_out itself):
 *
 *   d_y(p, :)            = weights[order[p]] * d_out(order[p] / topk, :),  zeros where order[p] is
 *                          outside [0, tokens * topk)
 *   d_weights[t*topk+j]  = sum over c of d_out(t, c) * y(slot[t*topk+j], c), 0 for a slot outside
 *                          [0, rows)
 *
 * in fp32 in a fixed order, rounded once; d_y has the type of y, d_weights that of the weights.
 * Either may be NULL (y is read for d_weights only).  Every row of d_y is written; it may not overlap
 * y or d_out. */
typedef struct combine_grad_args {
  const void* d_out;          /* tokens x cols, row stride ld_out                                   */
  const void* y;              /* rows x cols, row stride ldy; NULL without d_weights                */
  int32_t type, weight_type;
  int64_t tokens, rows, cols, ld_out, ldy;
  const int32_t* order;       /* `rows` values; NULL without d_y                                    */
  const int32_t* slot;        /* tokens * topk values                                               */
  const void* weights;        /* tokens * topk values; NULL without d_y                             */
  void* d_y;                  /* rows x cols, row stride ld_dy, or NULL                             */
  int64_t ld_dy;
  void* d_weights;            /* tokens * topk values, or NULL                                      */
  int32_t topk;
} combine_grad_args;
int route_combine_grad(const combine_grad_args* args, void* stream);

/* Errors of all: GEMM_ERR_INVALID_ARG, GEMM_ERR_DTYPE_COMBO, GEMM_ERR_LAYOUT,
 * GEMM_ERR_MISALIGNED, GEMM_ERR_ARCH, GEMM_ERR_HIP, GEMM_ERR_LAUNCH. */

#ifdef __cplusplus
}
#endif
#endif /* HTROUTE_H */
