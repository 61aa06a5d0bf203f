/*
 * expert_ops.h - C ABI of the expert-layer operators of libgemm_f32.so
 * (MI355X, gfx950): routing tokens to experts, products grouped by expert in
 * 32-bit and bfloat16 precision with their gradients, microscaled 4-bit and
 * 8-bit integer quantisation and products, and orthogonalised updates.
 *
 * Conventions, as in gemm_f32.h:
 *  - Return value: a gemm_f32_status code.  Nothing here throws, prints or
 *    aborts, allocates memory or synchronises; work is enqueued on `stream`
 *    (a hipStream_t; NULL = the null stream) and may be captured in a graph.
 *  - Pointers are device pointers of the current device, owned by the caller.
 *    Outputs overlap no other operand.  Operands of `dtype` EXPERT_F32 are
 *    4-byte, of EXPERT_BF16 2-byte aligned; int32 and float pointers, scales
 *    and the routings' workspace 4-byte, codes and the other workspaces 16-byte
 *    aligned.
 *  - Sizes and leading dimensions are in elements; sums, softmax statistics
 *    and products are held in 32 bits; a result of dtype EXPERT_BF16 is
 *    rounded once.  The same call on the same inputs gives the same bits.
 *  - Rows sorted by expert: expert e owns rows offsets[e] .. offsets[e + 1] of
 *    A and C.  offsets holds groups + 1 int32, not decreasing, within 0 .. m;
 *    it is read on the device, where values outside are clamped (wrong
 *    offsets give wrong results or leave rows of C as they were, and access
 *    nothing outside the operands).  Experts may be empty.  Rows before
 *    offsets[0] and from offsets[groups] on belong to no expert: their rows
 *    of C are zero.
 *  - m may be 0 (no rows); groups, n and k are at least 1; sizes are below
 *    2^31.  One row of a product's operand is below 8 MiB, an expert's matrix
 *    and C's tile rows in 32-bit precision below 2 GiB; the whole of A, B or C
 *    may be larger.  Counted in 32 bits, so below 2^31: of a product
 *    (m / 64 + 1) (groups + 2), with m / 16 where an expert has 16 rows or fewer
 *    on average, and (m / 16 + groups + 2) ceil(n / 32); of a 4-bit operand
 *    rows ceil(k / 32).  A matrix to quantise to 8 bits has up to 2^31 - 2049 columns.
 *  - A launch holds less than 2^32 threads, or the call is refused
 *    (GEMM_F32_ERR_INVALID_VALUE): a routing takes up to 2^29 - 128 tokens, its
 *    gradient 2^28 - 16; a 4-bit operand of rows of k columns has
 *    rows ceil(k / 512) up to 2^26 - 4; an 8-bit operand up to 2^26 - 4 rows of
 *    up to 2048 columns, 2^24 - 1 longer ones, rows ceil(k / 256) up to 2^26 - 4 back to
 *    values, and tiles of 16 x 16 below 2^23 where its experts have 16 rows or fewer; a
 *    product's tiles of 16 rows (up to 16
 *    rows an expert on average, else 64 or 128) and 32 to 128 columns, those
 *    of empty experts among them, are below 2^24.
 *  - Errors: GEMM_F32_ERR_INVALID_VALUE (an argument outside the above),
 *    GEMM_F32_ERR_NO_DEVICE, GEMM_F32_ERR_UNSUPPORTED_DEVICE,
 *    GEMM_F32_ERR_HIP (a launch failed; gemm_f32_last_hip_error),
 *    GEMM_F32_ERR_SCRATCH_TOO_SMALL (a workspace below the stated size).
 */
#ifndef EXPERT_OPS_H
#define EXPERT_OPS_H

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

enum expert_dtype {
    EXPERT_F32 = 0,
    EXPERT_BF16 = 1
};

/*
 * C_e = act(A_e . B_e + bias_e) for every expert e, A_e its rows of A.
 *   A: m x k, rows lda apart.  B: groups matrices expert_stride apart, each
 *   k x n with B(kk, j) = B[kk*ldb + j] (layout_b GEMM_F32_ROW_MAJOR) or
 *   B[j*ldb + kk] (GEMM_F32_COL_MAJOR).  C: m x n, rows ldc apart, of dtype.
 *   bias: groups x n floats (contiguous) or NULL.  activation: enum
 *   gemm_f32_activation.
 * The gradient with respect to A is the same call on the gradient of C with
 * B's layout exchanged.
 */
int expert_grouped_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *A, int64_t lda,
                          const void *B, int layout_b, int64_t ldb, int64_t expert_stride, const int *offsets,
                          const float *bias, int activation, void *C, int64_t ldc, void *stream);

/*
 * dB_e = A_e^T . G_e: A m x k, G m x n; dB: groups matrices k x n,
 * expert_stride apart, rows ldd apart, of dtype; zero for an empty expert.
 * The experts share no element: their matrices lie one after the other
 * (expert_stride >= (k - 1) ldd + n) or their rows in turn (expert_stride >= n,
 * ldd >= (groups - 1) expert_stride + n).
 * ceil(k / 64) ceil(n / 64), rounded up to a multiple of 8, times groups is
 * below 2^31.
 */
int expert_grouped_weight_grad(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *A, int64_t lda,
                               const void *G, int64_t ldg, const int *offsets, void *dB, int64_t ldd,
                               int64_t expert_stride, void *stream);

/*
 * Microscaled 4-bit floating point.  Blocks of 32 values along k share a
 * scale 2^e, e = max(floor(log2(largest magnitude)) - 2, -127), stored as the
 * byte 127 + e; a value is its sign and the nearest of 0, .5, 1, 1.5, 2, 3, 4,
 * 6 (codes 0 to 7, sign bit 8) to value / 2^e, ties to the even code,
 * saturating at 6.  A block with an infinity or a NaN gets the byte 255,
 * which stands for NaN.  With kp = k rounded up to 128: codes (rows, kp / 2)
 * bytes, the even column in the low half, zero past k; scales (kp / 128,
 * rows, 4) bytes, the four blocks of a row's 128 columns side by side.
 *
 * quantize reads X(r, c) = X[r*ld + c] (layout GEMM_F32_ROW_MAJOR) or
 * X[c*ld + r] (GEMM_F32_COL_MAJOR); dequantize writes X[r*ld + c].
 */
int expert_mx4_quantize(int dtype, int64_t rows, int64_t k, const void *X, int layout, int64_t ld, void *codes,
                        void *scales, void *stream);
int expert_mx4_dequantize(int dtype, int64_t rows, int64_t k, const void *codes, const void *scales, void *X,
                          int64_t ld, void *stream);

/*
 * Y_e = act(Q(X_e) . W_e^T + bias_e): X m x k of dtype is quantised as by
 * expert_mx4_quantize on the way, W_e is an n x k matrix held as codes
 * (groups, n, kp / 2) and scales (groups, kp / 128, n, 4); its codes past k are
 * zero.  offsets NULL: groups is 1 and W_0 takes every row.
 * workspace: expert_mx4_workspace bytes (may be 0: then NULL is allowed), free
 * for reuse when the call's work on the stream is done.
 */
int64_t expert_mx4_workspace(int64_t m, int64_t n, int64_t k, int64_t groups);
int expert_mx4_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *X, int64_t ldx,
                      const void *codes, const void *scales, const int *offsets, const float *bias, int activation,
                      void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Routing.  For each token the `choices` largest of its `groups` logits,
 * largest first, equal ones by the lower expert; logits of -inf or NaN are
 * never chosen (+inf is not supported: its weights are NaN).
 *   weights (tokens, choices) floats: softmax over the chosen logits
 *     (normalize 1) or over all of the token's (0), at the chosen ones;
 *   experts (tokens, choices) int32;
 *   offsets (groups + 1) int32 and order (tokens * choices) int32: the slots
 *     token * choices + j sorted by expert, equal ones in slot order; expert
 *     e's are order[offsets[e]] .. order[offsets[e + 1] - 1].
 * A slot for which no expert is left has expert -1 and weight 0 and is not in
 * order, whose places from offsets[groups] on hold -1.
 *   1 <= choices <= min(groups, 32), groups <= 1024, tokens >= 0,
 *   tokens * choices at most 2^31 - 2048.
 * workspace: expert_route_workspace bytes, as above.
 */
int64_t expert_route_workspace(int64_t tokens, int64_t groups);
int expert_route(int dtype, int64_t tokens, int64_t groups, int64_t choices, int normalize, const void *logits,
                 int64_t ld, float *weights, int *experts, int *offsets, int *order, void *workspace,
                 int64_t workspace_bytes, void *stream);

/*
 * dlogits = w (g - sum_j w_j g_j) over the experts the softmax of the same
 * expert_route call sums over; g, (tokens, choices) floats, is the gradient
 * with respect to its weights.  Zero elsewhere.
 */
int expert_route_grad(int dtype, int64_t tokens, int64_t groups, int64_t choices, int normalize, const void *logits,
                      int64_t ld, const float *weights, const int *experts, const float *grad, void *dlogits,
                      int64_t ldd, void *stream);

/*
 * Routing by scores, with a bias for balance and sets of experts.
 *   score s: sigmoid(logit), or softmax over the token's logits.
 *   key c = s + bias[expert] (bias NULL: 0), in 64 bits: what is chosen by.  An
 *   expert whose logit is -inf or NaN, or whose bias is -inf or NaN, is never
 *   chosen (+inf logits: not supported with softmax scores).
 *   The experts lie in `sets` sets of groups / sets neighbouring ones.  A set's
 *   value is the sum of its two largest keys (of one, where it has one); the
 *   `kept_sets` sets with the largest values stay, equal ones by the lower set.
 *   Chosen are the `choices` largest keys in them, equal ones by the lower
 *   expert.
 *   weights: scale s / (sum of the chosen s) (normalize 1; 0 where the sum is 0) or
 *   scale s (0), without the bias.
 * experts, offsets, order and the slots that find no expert: as expert_route.
 *   groups <= 1024, a multiple of sets; sets <= 64; 1 <= kept_sets <= sets;
 *   1 <= choices <= min(32, kept_sets groups / sets); scale > 0 and finite; tokens
 *   as for expert_route.
 * workspace: expert_route_balanced_workspace bytes.
 */
enum expert_scores {
    EXPERT_SIGMOID = 0,
    EXPERT_SOFTMAX = 1
};

int64_t expert_route_balanced_workspace(int64_t tokens, int64_t groups);
int expert_route_balanced(int dtype, int64_t tokens, int64_t groups, int64_t choices, int scores, int64_t sets,
                          int64_t kept_sets, int normalize, float scale, const void *logits, int64_t ld,
                          const float *bias, float *weights, int *experts, int *offsets, int *order, void *workspace,
                          int64_t workspace_bytes, void *stream);

/*
 * The logits' gradient from g, that of the weights of the same
 * expert_route_balanced call, (tokens, choices) floats; the choice and the bias
 * have none.  With dot = sum_j w_j g_j / scale over the token's slots (0 unless
 * normalize) a chosen expert's is w (g - dot) (1 - s) (sigmoid) or w (g - dot)
 * (softmax), another's 0; softmax without normalize adds -s sum_j w_j g_j to
 * every expert's.
 */
int expert_route_balanced_grad(int dtype, int64_t tokens, int64_t groups, int64_t choices, int scores, int normalize,
                               float scale, const void *logits, int64_t ld, const float *weights, const int *experts,
                               const float *grad, void *dlogits, int64_t ldd, void *stream);

/*
 * 8-bit integers with a scale for each row: scale = largest magnitude / 127,
 * code = the whole number nearest to x * (127 / largest magnitude), ties to
 * even, each step rounded in 32 bits.  A row whose largest magnitude is below
 * 2^-119 gets scale 0 and codes 0, one with an infinity or a NaN scale NaN and
 * codes 0.  With kp = k rounded up to 16: codes (rows, kp) bytes, zero past k;
 * scales (rows) floats.  quantize reads X as expert_mx4_quantize does; dequantize
 * writes X[r*ld + c] = codes * scale, rounded once.
 */
int expert_int8_quantize(int dtype, int64_t rows, int64_t k, const void *X, int layout, int64_t ld, void *codes,
                         float *scales, void *stream);
int expert_int8_dequantize(int dtype, int64_t rows, int64_t k, const void *codes, const float *scales, void *X,
                           int64_t ld, void *stream);

/*
 * Y_e = act(Q(X_e) . Q(W_e)^T + bias_e): X m x k of dtype is quantised on the way,
 * a scale for each row (token); W_e is held as n x kp codes, kp as above, and n
 * scales (a scale for each row, channel), the experts' one after the other.  The
 * sums of the codes' products are exact; times X's scale, times W's, plus bias,
 * each rounded in 32 bits.  k is at most 131072.  offsets NULL: groups is 1 and W_0
 * takes every row.
 * workspace: expert_int8_workspace bytes, free for reuse when the call's work on
 * the stream is done.
 */
int64_t expert_int8_workspace(int64_t m, int64_t k);
int expert_int8_linear(int dtype, int64_t m, int64_t n, int64_t k, int64_t groups, const void *X, int64_t ldx,
                       const void *codes, const float *scales, const int *offsets, const float *bias, int activation,
                       void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Y = scale * X orthogonalised, for each of `batch` matrices of rows x cols, rows
 * ldx (ldy) and matrices stride_x (stride_y) elements apart: X / |X| (2-norm of the
 * entries; a matrix of zeros stays one), then `steps` times, with A = X X^T and the
 * step's three coefficients a, b, c (in host memory, 3 * steps floats, read before
 * the call returns),
 *   X <- (a I + b A + c A A) X      (of a matrix with rows > cols its transposed),
 * which takes every singular value s to a s + b s^3 + c s^5.  X, A and a I + b A + c A A
 * are held in 22 bits between the products, whatever the type, sums in 32; a result of
 * dtype EXPERT_BF16 is rounded once.  Y may be X.
 *   steps 1 .. 64; coefficients that could let an entry of A, a I + b A + c A A or,
 *   before the last step, X pass 31 are refused; cols and rows below 2^22 - 64, and workgroups of 64 x 64
 *   in all below 2^24.
 * workspace: expert_orthogonalize_workspace bytes (for as many matrices at a time as
 * 2 GiB hold, one at least: about 8 bytes an entry, and of the smaller square 8; 128 MiB
 * more where their smaller squares have more than 256 blocks of 64 x 64 on and below the
 * diagonals).
 */
int64_t expert_orthogonalize_workspace(int dtype, int64_t batch, int64_t rows, int64_t cols);
int expert_orthogonalize(int dtype, int64_t batch, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                         int64_t stride_x, int steps, const float *coefficients, float scale, void *Y, int64_t ldy,
                         int64_t stride_y, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERT_OPS_H */
