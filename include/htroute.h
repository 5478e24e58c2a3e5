/*
 * htroute.h -- C ABI of the expert routing that stands before a grouped product: which rows go to
 * which expert, in the order and with the offsets that gemm_run_grouped and gemm_scaled_run take,
 * and the loss that keeps the experts evenly used, with its gradient.
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

/* Errors of all three: GEMM_ERR_INVALID_ARG, GEMM_ERR_DTYPE_COMBO, GEMM_ERR_LAYOUT,
 * GEMM_ERR_MISALIGNED, GEMM_ERR_ARCH, GEMM_ERR_HIP, GEMM_ERR_LAUNCH. */

#ifdef __cplusplus
}
#endif
#endif /* HTROUTE_H */
