/*
 * htscaled.h -- C ABI of the block-scaled e4m3 products and of the quantisation that feeds them.
 *
 * A block-scaled operand is an e4m3 matrix with one fp32 scale for each block of 128 values along
 * K: element (r, k) stands for q(r, k) * scale(r / rows_per_block, k / 128).  The products compute
 *
 *   D = act( alpha * row_scale[m] * sum over k of A(m, k) * B(n, k)  +  beta * C  +  bias[n] )
 *
 * with those values.  The sum over a block of k is multiplied by the two scales' product and added to
 * an fp32 accumulator, so a scale never has to be a power of two.  What a sum over a block keeps
 * depends on D's type:
 *
 *   fp32 D   products of codes are exact and added in fp32.
 *   bf16 D   an 8-bit matrix instruction adds the block, 8 neighbouring k (from a multiple of 8 on) at
 *            a time: with 2^E the largest product of their powers of two, each product loses what lies
 *            below 2^(E - 13), towards zero.  D before its rounding is within 2^-10 of the sum over k
 *            of |A(m, k) B(n, k)|, times |alpha row_scale[m]|; on random codes within 1.3e-5 to
 *            5.6e-5.  Where large products cancel, that can be more than a step of the result, and
 *            small products beside them can be lost whole: an fp32 D keeps them.
 *
 * Status codes, element types and activations are those of htgemm.h.  The caller owns every
 * device buffer and the stream; calls are asynchronous; the buffers and the stream belong to the
 * current device.  Nothing throws across this interface.
 */
#ifndef HTSCALED_H
#define HTSCALED_H

#include "htgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values of k (and, for 128 x 128 blocks, of n) that share a scale. */
#define GEMM_SCALED_BLOCK 128

/* What the descriptor's `batch` counts. */
enum {
  GEMM_SCALED_SINGLE = 0, /* one product; batch is 0 or 1                                          */
  GEMM_SCALED_BATCH = 1,  /* `batch` products of this shape at the *_l strides                     */
  GEMM_SCALED_ROWS = 2,   /* experts: group e owns rows [offsets[e], offsets[e+1]) of A, C and D   */
                          /* and multiplies them by B + e * b_stride_l                             */
  GEMM_SCALED_K = 3       /* experts' weight gradients: D + e * d_stride_l is the product over     */
                          /* the k in [offsets[e], offsets[e+1])                                   */
};

typedef struct gemm_scaled_desc {
  int64_t M, N, K;            /* A is M x K, B is N x K (both K-contiguous), D is M x N            */
  int32_t d_type;             /* GEMM_BF16 or GEMM_F32: the type of D, C and bias                  */
  int32_t b_block;            /* columns (rows of the N x K matrix) of B that share a scale: 128   */
                              /* (weights) or 1 (activations, gradients); A's scales are per row   */
  int64_t lda, ldb;           /* elements between rows of A (>= K) and of B (>= K)                 */
  int64_t ldc, ldd;           /* elements between rows of C and D (>= N); unit column stride       */
  int64_t a_scale_m, a_scale_k; /* scale of A(m, k) at a_scale[m * a_scale_m + (k/128) * a_scale_k] */
  int64_t b_scale_n, b_scale_k; /* of B(n, k) at b_scale[(n/b_block) * b_scale_n + (k/128) * b_scale_k] */
  int32_t has_c, has_bias, act, has_row_scale;
  int32_t form;               /* GEMM_SCALED_SINGLE, _BATCH, _ROWS or _K                           */
  int32_t split_k;            /* 0: the library decides, 1: never, 2..64: that many slices of k;   */
                              /* slices only with GEMM_SCALED_SINGLE                               */
  int64_t batch;              /* products or groups, 1..65535                                      */
  int64_t a_stride_l, b_stride_l, c_stride_l, d_stride_l; /* elements from one product to the next */
  int64_t a_scale_l, b_scale_l;                            /* the same for the scales               */
} gemm_scaled_desc;

typedef struct gemm_scaled_s* gemm_scaled_t;

/* Validate `desc` and choose a kernel.  Host only.  Errors: GEMM_ERR_INVALID_ARG (a negative or
 * too large size -- also of a launch, which has fewer than 2^32 threads --, an unknown enum, a split
 * of a batch or of groups, batch < 1 with a form that needs it, d_stride_l == 0 where products would
 * overwrite each other), GEMM_ERR_DTYPE_COMBO, GEMM_ERR_LAYOUT (a leading dimension below its row, a
 * negative stride), GEMM_ERR_ARCH, GEMM_ERR_HIP.
 *
 * Strides a form has no use for are ignored: a_stride_l, c_stride_l, d_stride_l and a_scale_l with
 * GEMM_SCALED_ROWS; a_stride_l, b_stride_l, a_scale_l and b_scale_l with GEMM_SCALED_K.  bias is
 * shared by the products or groups, row_scale too (with GEMM_SCALED_ROWS it has a value for each
 * of the M rows). */
int gemm_scaled_create(const gemm_scaled_desc* desc, gemm_scaled_t* out);

/* Bytes of device workspace a run needs (fp32 partial sums when k is split, else 0).  Its contents
 * after a run are unspecified; two runs in flight at once need two workspaces. */
int gemm_scaled_workspace_size(gemm_scaled_t h, size_t* bytes);

typedef struct gemm_scaled_args {
  const void* A;
  const float* a_scale;
  const void* B;
  const float* b_scale;
  const void* C;              /* read only when beta != 0                                           */
  void* D;
  const void* bias;           /* N values, non-NULL iff has_bias                                    */
  const float* row_scale;     /* M values, non-NULL iff has_row_scale                               */
  const int32_t* offsets;     /* batch + 1 device values for GEMM_SCALED_ROWS and _K, else NULL     */
  float alpha, beta;
  void* workspace;            /* gemm_scaled_workspace_size bytes, 16-byte aligned                  */
} gemm_scaled_args;

/* Enqueue the product on `stream`.  Pointers need the alignment of their elements; A and B are
 * read fastest when their bases, leading dimensions and batch strides are multiples of 16 bytes
 * and K is a multiple of 16 (quant_blocks pads rows with zeros for that; a K that counts them gives
 * the same sums), with single-byte loads otherwise (333 x 4096 x 8191: 620 us, x 8192: 28 us).  The
 * kernel of the largest bf16 products takes A's scales with a_scale_m == 1 and B's with b_block == 128;
 * other scale layouts of the same product run on smaller tiles (8192^3: 436 us, with a_scale_k == 1
 * 632, with b_block == 1 644).  M == 0 or N == 0 is a valid empty problem; K == 0 (or an empty group with
 * GEMM_SCALED_K) gives D = act(beta * C + bias).  beta == 0 reads no C.  D may be C itself, with
 * the same strides.  a_scale[m] * b_scale[n] is formed in fp32 and has to be a finite, normal
 * number for the block's products to be exact to fp32; a NaN scale makes its block's outputs NaN.
 *
 * offsets are read on the device.  They are clamped into [0, M] ([0, K] with GEMM_SCALED_K) and
 * made non-decreasing (offset e becomes the largest of offsets[0..e]); rows before the first and
 * behind the last are not written.  With GEMM_SCALED_K every offset is also rounded down to a
 * multiple of 128, except one that equals K, because a block of k has one scale.
 *
 * Errors: GEMM_ERR_BAD_HANDLE, GEMM_ERR_INVALID_ARG (a missing or a superfluous pointer, or 2^32 threads
 * and more of the kernel that these pointers' alignment needs), GEMM_ERR_MISALIGNED, GEMM_ERR_LAUNCH.
 * An error launches nothing. */
int gemm_scaled_run(gemm_scaled_t h, const gemm_scaled_args* args, void* stream);

/* Free a handle.  NULL is accepted. */
int gemm_scaled_destroy(gemm_scaled_t h);

/* What the handle chose for operands that the 16-byte loads can read. */
typedef struct gemm_scaled_info {
  int32_t bm, bn;             /* workgroup tile                                                     */
  int32_t waves;
  int32_t lds_bytes;
  int32_t split_k;            /* slices of k (1: none)                                              */
  int64_t grid;               /* workgroups per launch                                              */
  char name[64];
} gemm_scaled_info;
int gemm_scaled_get_info(gemm_scaled_t h, gemm_scaled_info* info);

/* ---- quantisation ------------------------------------------------------------------------- */
/* Rounds an f32, f16 or bf16 matrix to block-scaled e4m3, row-major, transposed, or both from one
 * read.  For a block with largest magnitude `top`:
 *
 *   t = max(top, 448 * 2^-126);  scale = t / 448;  q = e4m3(clamp(x * (448 / t), -448, 448))
 *
 * in fp32 with one rounding per operation, the conversion to nearest with ties to even.  With
 * pow2, scale is the least power of two (not below 2^-126) with top / scale <= 448, and
 * q = e4m3(x / scale), which then rounds once.  A block that holds a NaN or an infinity gets
 * scale NaN and every q 0x7f (NaN).
 *
 * Blocks: block_rows == 1 gives q a scale for each row and 128 columns, and qt (the transpose) a
 * scale for each column and 128 rows -- the two layouts a product and its weight gradient read.
 * block_rows == 128 gives both the scale of the 128 x 128 block. */
typedef struct quant_args {
  const void* x;              /* x_rows x cols (rows x cols without row_index), row stride ldx      */
  int32_t x_type;             /* GEMM_F32, GEMM_F16 or GEMM_BF16                                    */
  int32_t block_rows;         /* 1 or 128                                                           */
  int32_t pow2;               /* 1: scales are powers of two                                        */
  int32_t index_div;          /* >= 1: row r is x's row row_index[r] / index_div                    */
  int64_t rows, cols, ldx;
  const int32_t* row_index;   /* NULL, or `rows` device values; a value below 0 or at or above     */
  int64_t x_rows;             /* x_rows * index_div gives a row of zeros                             */
  void* q;                    /* rows x cols codes, row stride ldq >= cols, or NULL                 */
  int64_t ldq;
  float* scale;               /* of q(r, c) at scale[(r/block_rows) * scale_r + (c/128) * scale_c]  */
  int64_t scale_r, scale_c;
  void* qt;                   /* cols x rows codes, row stride ldqt >= rows, or NULL                */
  int64_t ldqt;
  float* scale_t;             /* block_rows == 1: of qt(c, r) at scale_t[c * scale_t_c +            */
  int64_t scale_t_c, scale_t_r; /* (r/128) * scale_t_r]; NULL with block_rows == 128 (scale serves) */
  int32_t pad;                /* 1: every row of q (qt) is continued with zeros to a multiple of 16 */
                              /* codes, or to ldq (ldqt) where that is less; 0: nothing but the     */
                              /* rows x cols codes is written                                       */
} quant_args;

/* Enqueue the quantisation on `stream`.  With block_rows == 1, q and scale come together, as do qt
 * and scale_t; with 128, scale is required.  Nothing else of the outputs' memory is written.
 * Errors: GEMM_ERR_INVALID_ARG (also when neither q nor qt is given), GEMM_ERR_DTYPE_COMBO,
 * GEMM_ERR_LAYOUT (also for scale strides by which blocks would share a scale's place: the larger has
 * to pass all that the smaller spans), GEMM_ERR_MISALIGNED, GEMM_ERR_ARCH, GEMM_ERR_HIP, GEMM_ERR_LAUNCH. */
int quant_blocks(const quant_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HTSCALED_H */
