/*
 * gemm_grouped.h -- products grouped by expert and products in 8-bit integers, the operators a
 * mixture-of-experts layer and an 8-bit layer of a large language model add to gemm.h.
 *
 * Conventions are those of gemm.h: row-major storage, leading dimensions in elements, DEVICE
 * pointers owned by the caller, calls asynchronous on `stream`, nothing allocated or kept, a
 * negative status and nothing enqueued for invalid arguments, and the same handle.
 *
 * Groups.  The M rows (tokens) are sorted by group (expert): group g owns the rows offsets[g]
 * .. offsets[g+1] - 1.  `offsets` is a DEVICE array of groups + 1 int64 values, read by the
 * kernels only, so that a router's result never has to reach the host.  A group may be empty.
 * Rows before offsets[0] or from offsets[groups] on belong to no group: they are neither read
 * nor written.  The kernels read each offset clamped to 0 .. M and raised to the largest one
 * before it, so that no content of the array makes a call touch anything outside the rows it was
 * given, and no two groups ever share a row.
 */
#ifndef TILED_GEMM_GROUPED_H
#define TILED_GEMM_GROUPED_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Kernels of the entry points below.  AUTO picks by type, layout, alignment and size. */
typedef enum gemm_grouped_kernel {
  GEMM_GROUPED_AUTO = 0,
  GEMM_GROUPED_ANY = 1, /* 64x64 tile, copies through registers: any alignment, layout and size */
  /* The tiles below copy 16-byte chunks: A, B (D) and C start on 16 bytes, the rows of A and B (D)
     and B's matrices follow each other at whole multiples of 16 bytes (at most 2^23 a row), the
     rows and matrices of C at multiples of 4 elements. */
  GEMM_GROUPED_MFMA_64 = 2,      /* 64x64 tile, the K loop split between two groups of waves */
  GEMM_GROUPED_MFMA_128 = 3,     /* 128x128 tile */
  GEMM_GROUPED_MFMA_256 = 4,     /* 256x256 tile, with 128x128 ones where rows or rounds end */
  GEMM_GROUPED_STREAM = 5,       /* few rows a group (decoding): weights streamed through registers,
                                    16 to 64 rows a tile, any alignment; rows of A and B of at most
                                    2^23 bytes, N >= 4 for a B stored K x N; not the gradient */
} gemm_grouped_kernel_t;

/* The product of each group's rows with the group's own matrix:
 *
 *     C[r] = epi(alpha * A[r] op(B_g) + beta * C[r] [+ bias_g])   for every row r of group g
 *
 * A is M x K (lda >= K).  B_g starts at B + g * stride_b and is stored K x N (ldb >= N) or, with
 * transB, N x K (ldb >= K); stride_b >= 0 (0: one matrix for all groups).  C is M x N.  bias is
 * fp32, groups x N, contiguous (NULL without GEMM_EPI_BIAS).  type: GEMM_F16 or GEMM_BF16, of
 * A, B and C; sums are fp32, rounded once.  Epilogue bits as gemm_run.  With the weights' other
 * transB, and C and A exchanged, the same call is the data gradient dA = dC op(B_g)^T.
 * Errors: as gemm_run (dimensions of at most 2^31 - 1024), plus GEMM_ERR_INVALID_VALUE for
 * groups < 0, stride_b < 0 or NULL offsets with groups > 0, and GEMM_ERR_UNSUPPORTED for groups >
 * 65535, for about 2^31 tiles of 64 x 64 or more (the most that any offsets can make of M rows; for
 * the streaming kernel, of 16 x 32, or x 64 for a B stored K x N), or for a kernel whose needs (see
 * gemm_grouped_kernel) do not hold.  M, N or groups of 0 enqueue nothing. */
GEMM_API gemm_status_t gemm_run_grouped(gemm_handle_t h, gemm_grouped_kernel_t kernel,
                                        void* stream, int64_t groups, const int64_t* offsets,
                                        int64_t M, int64_t N, int64_t K, int transB, float alpha,
                                        const void* A, int64_t lda, const void* B, int64_t ldb,
                                        int64_t stride_b, float beta, void* C, int64_t ldc,
                                        gemm_dtype_t type, uint32_t epilogue, const float* bias);

/* The weight and bias gradients of gemm_run_grouped:
 *
 *     C_g = alpha * A_g^T D_g + beta * C_g          (stored K x N; with transB, N x K)
 *     dbias_g[n] = sum over the group's rows r of D[r][n]          (NULL: not computed)
 *
 * A is M x K (lda >= K), the forward's input; D is M x N (ldd >= N), the gradient of its output.
 * C_g starts at C + g * stride_c; the matrices follow each other (stride_c of at least a matrix's
 * extent) or lie side by side (stride_c of at least a row's elements, all groups within ldc).
 * dbias is fp32, groups x N, contiguous.  type (of A and D): GEMM_F16 or GEMM_BF16; c_type: the
 * same, or GEMM_F32.  Sums are fp32, in an order that depends on the sizes only.  An empty group
 * gives beta * C_g and a zero dbias_g.  Errors: as gemm_run_grouped (the tiles are those of all
 * groups' gradients), with GEMM_ERR_INVALID_VALUE for any other stride_c.  With M = 0 every group
 * is empty. */
GEMM_API gemm_status_t gemm_run_grouped_wgrad(gemm_handle_t h, gemm_grouped_kernel_t kernel,
                                              void* stream, int64_t groups,
                                              const int64_t* offsets, int64_t M, int64_t N,
                                              int64_t K, int transB, float alpha, const void* A,
                                              int64_t lda, const void* D, int64_t ldd, float beta,
                                              void* C, int64_t ldc, int64_t stride_c,
                                              gemm_dtype_t type, gemm_dtype_t c_type,
                                              float* dbias);

/* The product of 8-bit integers (two's complement, -128 .. 127) with a scale for each row of A
 * (token) and each column of B (channel):
 *
 *     C[i][j] = epi(alpha * sa[i] * sb[j] * sum_k A[i][k] B[k][j] + beta * C[i][j] [+ bias[j]])
 *
 * A is M x K (lda >= K), B is stored K x N (ldb >= N) or, with transB, N x K (ldb >= K); sa is
 * fp32[M], sb fp32[N].  The integer sum is exact: K <= 131071, so that K * 128 * 128 < 2^31
 * (GEMM_ERR_UNSUPPORTED above).  It is scaled in fp32 as (sum * (alpha * sa[i])) * sb[j] and
 * rounded once to c_type: GEMM_F16, GEMM_BF16 or GEMM_F32.  Errors as gemm_run_grouped. */
GEMM_API gemm_status_t gemm_run_i8(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream,
                                   int64_t M, int64_t N, int64_t K, int transB, float alpha,
                                   const int8_t* A, int64_t lda, const float* sa,
                                   const int8_t* B, int64_t ldb, const float* sb, float beta,
                                   void* C, int64_t ldc, gemm_dtype_t c_type, uint32_t epilogue,
                                   const float* bias);

/* gemm_run_i8 by group: the rows of group g take B_g (as in gemm_run_grouped) with the column
 * scales sb[g * N ..] and the bias bias[g * N ..]; sa has one scale per row of A. */
GEMM_API gemm_status_t gemm_run_grouped_i8(gemm_handle_t h, gemm_grouped_kernel_t kernel,
                                           void* stream, int64_t groups, const int64_t* offsets,
                                           int64_t M, int64_t N, int64_t K, int transB,
                                           float alpha, const int8_t* A, int64_t lda,
                                           const float* sa, const int8_t* B, int64_t ldb,
                                           int64_t stride_b, const float* sb, float beta, void* C,
                                           int64_t ldc, gemm_dtype_t c_type, uint32_t epilogue,
                                           const float* bias);

/* Rows in 8-bit integers with a scale each, the A and sa of the products above:
 *
 *     scales[i] = max over k of |X[i][k]| / 127              (fp32, rounded to nearest even)
 *     Q[i][k]   = X[i][k] / scales[i], exactly, rounded to the nearest integer, ties to even
 *
 * X is M x K (ldx >= K) of x_type GEMM_F32, GEMM_F16 or GEMM_BF16; Q is M x K (ldq >= K).  The
 * codes lie in -127 .. 127 (clamped there: a scale that is a subnormal number may have been
 * rounded down).  A row of zeros (or whose scale underflows to 0) gives scale 0 and
 * codes 0; a row that holds a NaN gives scale NaN, one that holds an infinity and no NaN scale
 * infinity, both with codes 0, so that the row's products come out NaN.  K = 0 gives scales 0.
 * Errors as gemm_run (GEMM_ERR_ALIAS when Q or scales overlap X or each other). */
GEMM_API gemm_status_t gemm_quantize_rows(gemm_handle_t h, void* stream, int64_t M, int64_t K,
                                          const void* X, int64_t ldx, gemm_dtype_t x_type,
                                          int8_t* Q, int64_t ldq, float* scales);

/* Check the arguments of the calls above without touching any device.  gemm_check_args_grouped
 * serves gemm_run_grouped (b_type = c_type = type, sa and sb NULL), gemm_run_grouped_i8 and,
 * with groups = 1 and offsets NULL, gemm_run_i8 (i8 != 0: type is ignored). */
GEMM_API gemm_status_t gemm_check_args_grouped(int64_t groups, const int64_t* offsets, int64_t M,
                                               int64_t N, int64_t K, int transB, const void* A,
                                               int64_t lda, const float* sa, const void* B,
                                               int64_t ldb, int64_t stride_b, const float* sb,
                                               const void* C, int64_t ldc, int i8,
                                               gemm_dtype_t type, gemm_dtype_t c_type,
                                               uint32_t epilogue, const float* bias);
GEMM_API gemm_status_t gemm_check_args_grouped_wgrad(int64_t groups, const int64_t* offsets,
                                                     int64_t M, int64_t N, int64_t K, int transB,
                                                     const void* A, int64_t lda, const void* D,
                                                     int64_t ldd, const void* C, int64_t ldc,
                                                     int64_t stride_c, gemm_dtype_t type,
                                                     gemm_dtype_t c_type, const float* dbias);
GEMM_API gemm_status_t gemm_check_args_quantize_rows(int64_t M, int64_t K, const void* X,
                                                     int64_t ldx, gemm_dtype_t x_type,
                                                     const int8_t* Q, int64_t ldq,
                                                     const float* scales);

#ifdef __cplusplus
}
#endif

#endif /* TILED_GEMM_GROUPED_H */
