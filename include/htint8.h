/*
 * htint8.h -- C ABI of the products in 8-bit integers with a scale for each token and each channel,
 * and of the quantisation that feeds them.
 *
 *   D = act( (S(m, n) * (alpha * a_scale[m])) * b_scale[n]  +  beta * C  +  bias[n] )
 *   S(m, n) = sum over k of A(m, k) * B(n, k)
 *
 * A and B hold signed 8-bit codes; S is exact (32-bit integers, K <= GEMM_INT8_MAX_K) and is rounded
 * to fp32 once; the steps behind it are fp32, in the order above, with one rounding each at most; D
 * is rounded once more.  An output's bits depend neither on how k is split nor on the kernel.
 *
 * Status codes, element types and activations are those of htgemm.h.  The caller owns every
 * device buffer and the stream; calls are asynchronous; the buffers and the stream belong to the
 * current device.  Nothing throws across this interface.
 */
#ifndef HTINT8_H
#define HTINT8_H

#include "htgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The longest K: 131071 products of -128 and -128 still fit 32 bits. */
#define GEMM_INT8_MAX_K 131071

/* What the descriptor's `batch` counts. */
enum {
  GEMM_INT8_SINGLE = 0,       /* one product; batch is 0 or 1                                      */
  GEMM_INT8_BATCH = 1,        /* `batch` products of this shape at the *_l strides                 */
  GEMM_INT8_ROWS = 2          /* experts: group e owns rows [offsets[e], offsets[e+1]) of A, C and */
                              /* D and multiplies them by B + e * b_stride_l                       */
};

typedef struct gemm_int8_desc {
  int64_t M, N, K;            /* A is M x K, B is N x K (both K-contiguous), D is M x N            */
  int32_t d_type;             /* GEMM_BF16, GEMM_F16 or GEMM_F32: the type of D, C and bias        */
  int32_t form;               /* GEMM_INT8_SINGLE, _BATCH or _ROWS                                 */
  int64_t lda, ldb;           /* codes between rows of A (>= K) and of B (>= K)                    */
  int64_t ldc, ldd;           /* elements between rows of C and D (>= N); unit column stride       */
  int32_t has_c, has_bias, act;
  int32_t split_k;            /* 0: the library decides, 1: never, 2..64: that many slices of k;   */
                              /* slices only with GEMM_INT8_SINGLE                                 */
  int64_t batch;              /* products or groups, 1..65535                                      */
  int64_t a_stride_l, b_stride_l, c_stride_l, d_stride_l; /* elements from one product to the next */
  int64_t a_scale_l, b_scale_l;                            /* the same for the scales               */
} gemm_int8_desc;

typedef struct gemm_int8_s* gemm_int8_t;

/* Validate `desc` and choose a kernel.  Host only.  Errors: GEMM_ERR_INVALID_ARG (a negative or
 * too large size -- also of a launch, which has fewer than 2^32 threads along a dimension --, an
 * unknown enum, a split of a batch or of groups, batch < 1 with a form that needs it, d_stride_l == 0
 * where products would overwrite each other), GEMM_ERR_DTYPE_COMBO, GEMM_ERR_LAYOUT (a leading
 * dimension below its row, a negative stride), GEMM_ERR_ARCH, GEMM_ERR_HIP.
 *
 * With GEMM_INT8_ROWS a_stride_l, c_stride_l, d_stride_l and a_scale_l are ignored.  bias is shared
 * by the products or groups. */
int gemm_int8_create(const gemm_int8_desc* desc, gemm_int8_t* out);

/* Bytes of device workspace a run needs (32-bit partial sums when k is split, else 0).  Its contents
 * after a run are unspecified; two runs in flight at once need two workspaces. */
int gemm_int8_workspace_size(gemm_int8_t h, size_t* bytes);

typedef struct gemm_int8_args {
  const void* A;
  const float* a_scale;       /* M values                                                          */
  const void* B;
  const float* b_scale;       /* N values                                                          */
  const void* C;              /* read only when beta != 0                                          */
  void* D;
  const void* bias;           /* N values; NULL without has_bias (and, without N, with it)         */
  const int32_t* offsets;     /* batch + 1 device values for GEMM_INT8_ROWS, else NULL             */
  float alpha, beta;
  void* workspace;            /* gemm_int8_workspace_size bytes, 16-byte aligned                   */
} gemm_int8_args;

/* Enqueue the product on `stream`.  Pointers need the alignment of their elements.  A and B are
 * read fastest when their bases, leading dimensions and batch strides are multiples of 16 bytes, for
 * any K: what lies between the rows is not used, though the up to 15 bytes behind K that share its
 * last 16 are read.  Other rows take kernels that load at any byte.  M == 0 or N == 0 is a valid
 * empty problem; K == 0 gives D = act(beta * C + bias) and reads no scale.  beta == 0 reads no C.  D
 * may be C itself, with the same strides.  A NaN scale makes its row's or column's outputs NaN.
 *
 * offsets are read on the device.  They are clamped into [0, M] and made non-decreasing (offset e
 * becomes the largest of offsets[0..e]); rows before the first and behind the last are not written.
 *
 * Errors: GEMM_ERR_BAD_HANDLE, GEMM_ERR_INVALID_ARG (a missing or a superfluous pointer, or 2^32
 * threads and more of the kernel that these pointers' alignment needs), GEMM_ERR_MISALIGNED,
 * GEMM_ERR_LAUNCH.  An error launches nothing. */
int gemm_int8_run(gemm_int8_t h, const gemm_int8_args* args, void* stream);

/* Free a handle.  NULL is accepted. */
int gemm_int8_destroy(gemm_int8_t h);

/* What the handle chose for operands whose bases lie on 16 bytes. */
typedef struct gemm_int8_info {
  int32_t bm, bn;             /* workgroup tile                                                    */
  int32_t waves;
  int32_t lds_bytes;
  int32_t split_k;            /* slices of k (1: none)                                             */
  int64_t grid;               /* workgroups per launch                                             */
  char name[64];
} gemm_int8_info;
int gemm_int8_get_info(gemm_int8_t h, gemm_int8_info* info);

/* ---- quantisation ------------------------------------------------------------------------- */
/* Rounds the rows of an f32, f16 or bf16 matrix to 8-bit codes with one scale each:
 *
 *   t = max(largest |x| of the row, 127 * 2^-126);  scale = t / 127;
 *   q = clamp(rint(x * (127 / t)), -127, 127)
 *
 * in fp32 with one rounding for each operation, rint to the nearest with ties to even.  A row that
 * holds a NaN or an infinity gets scale NaN and codes of zero, so that a product's outputs of that
 * row are NaN.  With `gate`, x is act(gate) * x, element by element in fp32, as between the two
 * products of a gated layer. */
typedef struct quant_rows_args {
  const void* x;              /* x_rows x cols (rows x cols without row_index), row stride ldx      */
  const void* gate;           /* NULL, or a matrix of the same type and shape, row stride ldg       */
  int32_t x_type;             /* GEMM_F32, GEMM_F16 or GEMM_BF16                                    */
  int32_t act;                /* the gate's activation; GEMM_ACT_NONE without one                   */
  int64_t rows, cols, ldx, ldg;
  const int32_t* row_index;   /* NULL, or `rows` device values: row r is x's (and gate's) row       */
  int64_t x_rows;             /* row_index[r] / index_div; a value below 0 or at or above           */
  int32_t index_div;          /* x_rows * index_div gives a row of zeros.  index_div >= 1           */
  int32_t pad;                /* 1: every row of q is continued with zeros to a multiple of 16      */
                              /* codes, or to ldq where that is less; 0: nothing but the rows x     */
                              /* cols codes is written                                              */
  void* q;                    /* rows x cols codes, row stride ldq >= cols                          */
  int64_t ldq;
  float* scale;               /* rows values                                                        */
} quant_rows_args;

/* Enqueue the quantisation on `stream`.  Errors: GEMM_ERR_INVALID_ARG (also a row of more than 2^24
 * values), GEMM_ERR_DTYPE_COMBO, GEMM_ERR_LAYOUT, GEMM_ERR_MISALIGNED, GEMM_ERR_ARCH, GEMM_ERR_HIP,
 * GEMM_ERR_LAUNCH.  rows == 0 is a valid empty problem, and so is cols == 0 (which writes the scale of
 * rows of zeros).  q and scale may not overlap x, gate or row_index. */
int quant_rows(const quant_rows_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HTINT8_H */
