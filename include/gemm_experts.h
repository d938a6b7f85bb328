/*
 * gemm_experts.h -- the way of tokens to their experts and back, and products by expert in MXFP4: what
 * a mixture-of-experts layer needs next to the grouped products of gemm_grouped.h.
 *
 * Conventions are those of gemm.h: row-major storage, leading dimensions in elements, DEVICE pointers
 * owned by the caller, calls asynchronous on `stream`, nothing allocated or kept, a negative status and
 * nothing enqueued for invalid arguments, and the same handle.  A result that overlaps an operand or
 * another result is GEMM_ERR_ALIAS.  Dimensions of more than 2^31 - 1024, rows of more than 2^31 - 1024
 * (token, expert) pairs among them, are GEMM_ERR_UNSUPPORTED.
 *
 * A layer of E experts, `top` of them for each of T tokens:
 *
 *     gemm_route           logits -> expert, weight, place (T x top) and offsets (E + 1)
 *     gemm_dispatch_rows   the tokens' rows into the experts' order
 *       or gemm_quantize_mx, which writes them there in MXFP4
 *     gemm_run_grouped, gemm_run_grouped_i8 or gemm_run_grouped_mx with these offsets
 *     gemm_combine_rows    each token's answers, weighted, back into its row
 *
 * and, in training, gemm_combine_rows_grad, the gradients of the products, gemm_combine_rows without
 * weights (the gradient of dispatch) and gemm_route_grad.  No result has to reach the host.
 */
#ifndef TILED_GEMM_EXPERTS_H
#define TILED_GEMM_EXPERTS_H

#include "gemm_grouped.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What the logits of a token become: s = softmax over its experts, or the sigmoid of each. */
typedef enum gemm_score {
  GEMM_SCORE_SOFTMAX = 0,
  GEMM_SCORE_SIGMOID = 1
} gemm_score_t;

/* Workspace bytes gemm_route needs: 0 for up to 64 tokens of up to 128 experts (32 of up to 256, 16 of
 * more).  A negative status for sizes that gemm_route refuses.  Touches no device. */
GEMM_API int64_t gemm_route_workspace_bytes(int64_t tokens, int64_t experts);

/* The experts of each token and the order of the rows that go to them.
 *
 * logits: tokens x experts (ldl >= experts), x_type GEMM_F32, GEMM_F16 or GEMM_BF16; experts of 1 to
 * 1024, top of 1 to min(experts, 32).  With x the logits of a token and s its scores:
 *
 *     key[e]    = x[e], or with bias (fp32, one for each expert) s[e] + bias[e]
 *     expert[j] = the expert with the j-th largest key, the lower one of equal keys
 *     weight[j] = scale * s[expert[j]],                       or with renorm
 *                 scale * s[expert[j]] / (the sum of the chosen s)
 *
 * The bias decides the choice only.  Keys are compared as if computed in 64 bits.  Weights are fp32 sums
 * and quotients, each within (32 + |x - m|) 2^-24 of itself, x the expert's logit and m the token's largest;
 * a score under 2^-125 (with renorm, of the largest chosen score) may count as 0.
 *
 * Limited groups: the experts lie in `groups` runs of equal length (groups divides experts, at most
 * 64); a run is worth the sum of its group_top (1 or 2) largest keys (without a bias and with group_top
 * 2, of its largest s), and only the top_groups best runs count, the lower one of equal runs.  groups =
 * top_groups = group_top = 1: no limit.  top <= top_groups * experts / groups.
 *
 * What is not there: an expert whose logit or bias is -infinity is never chosen, and a run of such
 * experts neither.  Where a token has fewer than top experts left (a padded token: none), the rest of
 * its slots hold expert -1, weight 0 and place -1.  A key that is NaN counts as +infinity, so that a
 * token of NaN is answered with NaN and not with silence.  A softmax with NaN or +infinity among its
 * logits has no scores: the weights of all of the token's experts are NaN.
 *
 * place[t * top + j] is the row of the pair (t, j) when all pairs are sorted by expert and, within an
 * expert, by token; offsets[e] (int64, experts + 1) the row where expert e's start, offsets[experts]
 * their number: the groups of gemm_grouped.h.  expert, weight, place: tokens x top, contiguous.
 *
 * workspace: gemm_route_workspace_bytes(tokens, experts) bytes or more, any content, 16-byte aligned
 * (NULL where that is 0).  Calls that share one must not overlap (one stream, or synchronised).
 * Errors: GEMM_ERR_INVALID_VALUE for sizes that do not go together as above, ldl < experts, a NULL
 * pointer, an unknown score, renorm not 0 or 1, or a workspace that is NULL, too small or not aligned;
 * GEMM_ERR_UNSUPPORTED for other types, more than 2^29 tokens, more than 1024 experts, top over 32 or
 * groups over 64.  With no tokens the offsets are 0 and nothing else is written. */
GEMM_API gemm_status_t gemm_route(gemm_handle_t h, void* stream, int64_t tokens, int64_t experts,
                                  int64_t top, const void* logits, int64_t ldl, gemm_dtype_t x_type,
                                  gemm_score_t score, const float* bias, int64_t groups,
                                  int64_t top_groups, int group_top, int renorm, float scale,
                                  int32_t* expert, float* weight, int32_t* place, int64_t* offsets,
                                  void* workspace, int64_t workspace_bytes);

/* The gradient of the logits from that of gemm_route's weights (the choice itself has none):
 *
 *     dlogits[t][e] = sum over j of dweight[t][j] * d weight[t][j] / d x[t][e]
 *
 * logits, score, renorm and scale as gemm_route was given them, expert as it wrote them (the experts of
 * a token are distinct; -1 and any other number that is no expert is skipped); dweight fp32, tokens x
 * top; dlogits: tokens x experts (ldd >= experts) of x_type, computed in fp32 and rounded once.  Every
 * element is written.  A logit of -infinity has gradient 0, also where all of a token's are.  NaN or
 * +infinity among the logits of a softmax makes all of the token's gradients NaN; with renorm, where only
 * the chosen logits are read, those of the chosen if it is one of them, and the others stay 0.  Errors as
 * gemm_route. */
GEMM_API gemm_status_t gemm_route_grad(gemm_handle_t h, void* stream, int64_t tokens, int64_t experts,
                                       int64_t top, const void* logits, int64_t ldl, gemm_dtype_t x_type,
                                       gemm_score_t score, int renorm, float scale,
                                       const int32_t* expert, const float* dweight, void* dlogits,
                                       int64_t ldd);

/* Rows to the experts: A[place[t * top + j]] = X[t], for all j < top.
 * X is tokens x K (ldx >= K), A rows x K (lda >= K), both of type GEMM_F32, GEMM_F16 or GEMM_BF16.
 * A place outside 0 .. rows - 1 is skipped; rows of A that no pair has are left as they were.  Places
 * are distinct (gemm_route's are): a row that has two pairs holds parts of either's.  top >= 1, rows >= 0. */
GEMM_API gemm_status_t gemm_dispatch_rows(gemm_handle_t h, void* stream, int64_t tokens, int64_t top,
                                          int64_t K, const void* X, int64_t ldx, gemm_dtype_t type,
                                          const int32_t* place, int64_t rows, void* A, int64_t lda);

/* Rows back from the experts:
 *
 *     C[t] = sum over j of weight[t * top + j] * Y[place[t * top + j]]  +  beta * C[t]
 *
 * Y is rows x K (ldy >= K), C tokens x K (ldc >= K); weight fp32, or NULL for weights of 1 (the gradient
 * of gemm_dispatch_rows).  A place outside 0 .. rows - 1 adds nothing, whatever its weight.  Sums are
 * fp32 in the order of j, rounded once.  beta = 0: C is not read. */
GEMM_API gemm_status_t gemm_combine_rows(gemm_handle_t h, void* stream, int64_t tokens, int64_t top,
                                         int64_t K, const void* Y, int64_t ldy, gemm_dtype_t type,
                                         const int32_t* place, int64_t rows, const float* weight,
                                         float beta, void* C, int64_t ldc);

/* The gradients of gemm_combine_rows from D (tokens x K, ldd >= K), the gradient of C:
 *
 *     dY[place[t * top + j]]  = weight[t * top + j] * D[t]                      (rows x K, lddy >= K)
 *     dweight[t * top + j]    = sum over k of D[t][k] * Y[place[t * top + j]][k]         (fp32)
 *
 * A skipped place has dweight 0; rows of dY that no pair has are left as they were; places are distinct, as
 * for gemm_dispatch_rows.  dweight's sums are fp32, in an order that depends on K only. */
GEMM_API gemm_status_t gemm_combine_rows_grad(gemm_handle_t h, void* stream, int64_t tokens, int64_t top,
                                              int64_t K, const void* D, int64_t ldd, const void* Y,
                                              int64_t ldy, gemm_dtype_t type, const int32_t* place,
                                              int64_t rows, const float* weight, void* dY, int64_t lddy,
                                              float* dweight);

/* Rows in MXFP4, the operands of gemm_run_mx and gemm_run_grouped_mx: every run of 32 elements of a
 * row shares the power of two
 *
 *     e = floor(log2(max |x|)) - 2, at least -127          (OCP MX: the largest 4-bit magnitude is 6 =
 *                                                           1.5 * 2^2)
 *
 * stored as the byte e + 127, and holds x / 2^e rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
 * ties to the even code, at most 6, with x's sign.  A run of zeros has byte 0; one that holds an
 * infinity or a NaN has byte 255 (NaN) and codes 0, so that the row's products come out NaN.
 *
 * X is M x K (ldx >= K) of x_type GEMM_F32, GEMM_F16 or GEMM_BF16, K a multiple of 32; q_type is
 * GEMM_E2M1: Q has rows of ldq elements (two a byte, ldq even and at least K), S rows of lds >= K / 32
 * bytes.  With place NULL row i goes to row i (top 1, rows = M); with place (M x top, as gemm_route
 * writes it) to the rows place[i * top + j], as gemm_dispatch_rows would send it (distinct, too). */
GEMM_API gemm_status_t gemm_quantize_mx(gemm_handle_t h, void* stream, int64_t M, int64_t K,
                                        const void* X, int64_t ldx, gemm_dtype_t x_type, int64_t top,
                                        const int32_t* place, int64_t rows, void* Q, int64_t ldq,
                                        gemm_dtype_t q_type, uint8_t* S, int64_t lds);

/* The product of each group's rows with the group's own matrix, both in MXFP4:
 *
 *     C[r] = epi(alpha * A[r] B_g^T + beta * C[r] [+ bias_g])   for every row r of group g
 *
 * A is M x K (lda >= K) with scale bytes sa (M rows of ldsa >= K / 32); B_g starts stride_b elements
 * after B_(g-1), is stored N x K (ldb >= K) and has scale bytes at sb + g * stride_sb (N rows of ldsb >=
 * K / 32); type is GEMM_E2M1 (elements and scales as in gemm_run_mx); K is a multiple of 32, lda, ldb
 * and stride_b are even, stride_b and stride_sb >= 0 (0: one matrix for all groups).  C is M x N of
 * c_type GEMM_BF16, GEMM_F16 or GEMM_F32; bias fp32, groups x N.  Groups, offsets, epilogue, limits and
 * errors as gemm_run_grouped; with groups = 1, offsets may be NULL: one group has all rows (M = 1: one
 * token's matrix-vector product).
 *
 * Kernels: GEMM_GROUPED_STREAM (16 to 64 rows a tile, any alignment; rows of at most 2^23 bytes), and
 * GEMM_GROUPED_MFMA_64, _128 and _256, which need A, B, sa, sb and C on 16 bytes, lda, ldb and stride_b
 * multiples of 32, ldsa, ldsb and stride_sb of 16, ldc of 4, and less than 2^32 bytes of scales to a
 * group.  AUTO takes the tiles where they fit and pay.  GEMM_GROUPED_ANY is not among them
 * (GEMM_ERR_UNSUPPORTED). */
GEMM_API gemm_status_t gemm_run_grouped_mx(gemm_handle_t h, gemm_grouped_kernel_t kernel, void* stream,
                                           int64_t groups, const int64_t* offsets, int64_t M, int64_t N,
                                           int64_t K, float alpha, const void* A, int64_t lda,
                                           const uint8_t* sa, int64_t ldsa, const void* B, int64_t ldb,
                                           int64_t stride_b, const uint8_t* sb, int64_t ldsb,
                                           int64_t stride_sb, float beta, void* C, int64_t ldc,
                                           gemm_dtype_t type, gemm_dtype_t c_type, uint32_t epilogue,
                                           const float* bias);

/* Check the arguments of the calls above without touching any device. */
GEMM_API gemm_status_t gemm_check_args_route(int64_t tokens, int64_t experts, int64_t top,
                                             const void* logits, int64_t ldl, gemm_dtype_t x_type,
                                             gemm_score_t score, const float* bias, int64_t groups,
                                             int64_t top_groups, int group_top, int renorm,
                                             const int32_t* expert, const float* weight,
                                             const int32_t* place, const int64_t* offsets,
                                             const void* workspace, int64_t workspace_bytes);
GEMM_API gemm_status_t gemm_check_args_route_grad(int64_t tokens, int64_t experts, int64_t top,
                                                  const void* logits, int64_t ldl, gemm_dtype_t x_type,
                                                  gemm_score_t score, int renorm, const int32_t* expert,
                                                  const float* dweight, const void* dlogits, int64_t ldd);
GEMM_API gemm_status_t gemm_check_args_dispatch_rows(int64_t tokens, int64_t top, int64_t K,
                                                     const void* X, int64_t ldx, gemm_dtype_t type,
                                                     const int32_t* place, int64_t rows, const void* A,
                                                     int64_t lda);
GEMM_API gemm_status_t gemm_check_args_combine_rows(int64_t tokens, int64_t top, int64_t K, const void* Y,
                                                    int64_t ldy, gemm_dtype_t type, const int32_t* place,
                                                    int64_t rows, const float* weight, const void* C,
                                                    int64_t ldc);
GEMM_API gemm_status_t gemm_check_args_combine_rows_grad(int64_t tokens, int64_t top, int64_t K,
                                                         const void* D, int64_t ldd, const void* Y,
                                                         int64_t ldy, gemm_dtype_t type,
                                                         const int32_t* place, int64_t rows,
                                                         const float* weight, const void* dY,
                                                         int64_t lddy, const float* dweight);
GEMM_API gemm_status_t gemm_check_args_quantize_mx(int64_t M, int64_t K, const void* X, int64_t ldx,
                                                   gemm_dtype_t x_type, int64_t top, const int32_t* place,
                                                   int64_t rows, const void* Q, int64_t ldq,
                                                   gemm_dtype_t q_type, const uint8_t* S, int64_t lds);
GEMM_API gemm_status_t gemm_check_args_grouped_mx(int64_t groups, const int64_t* offsets, int64_t M,
                                                  int64_t N, int64_t K, const void* A, int64_t lda,
                                                  const uint8_t* sa, int64_t ldsa, const void* B,
                                                  int64_t ldb, int64_t stride_b, const uint8_t* sb,
                                                  int64_t ldsb, int64_t stride_sb, const void* C,
                                                  int64_t ldc, gemm_dtype_t type, gemm_dtype_t c_type,
                                                  uint32_t epilogue, const float* bias);

#ifdef __cplusplus
}
#endif

#endif /* TILED_GEMM_EXPERTS_H */
