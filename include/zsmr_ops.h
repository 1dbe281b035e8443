/*
 * zsmr_ops.h -- the operators around the shard step, in libzsmr.so (gfx950).
 *
 * A ZeRO step starts from 16-bit gradient rows and, where training clips, from
 * the norm of the whole reduced gradient.  This header has both ends of that:
 *   - the embedding lookup from the 16-bit working copy, and its gradient by
 *     sorted tokens into a rank's 16-bit gradient row;
 *   - the softmax cross entropy of the output head over a large vocabulary,
 *     whose logits are never kept, and its gradients;
 *   - the global gradient norm over many tensors, and clipping in place or
 *     into the flat 16-bit gradient row ("ZeRO and FSDP", ZeroAdam._flatten);
 *   - the clipped shard step: reduce with the shard's sum of squares, the join
 *     of all ranks' sums, and Adam on the clipped gradient with the cast
 *     ("The four schemes", Base._adam and ZeRO1.step).  The pages do not clip;
 *     the arithmetic of reduce, Adam and cast is that of zsmr.h;
 *   - the orthogonalised update of matrices by Newton-Schulz products, and the
 *     shard step that applies it to matrices a rank owns whole (reduce, momentum,
 *     orthogonalise, update, cast);
 *   - scores of logits that a program has: log probabilities of given tokens with
 *     entropy and top alternatives, and their gradient.
 *
 * The conventions of zsmr.h hold: status codes, caller-owned device memory,
 * asynchronous launches on the caller's stream, every argument checked before
 * anything is launched.  Further:
 *   - A workspace is device memory of at least the bytes the *_workspace call
 *     names, 16-byte aligned, with any content.  Calls on one stream may share
 *     it; calls that may run at the same time may not.
 *   - Inputs and outputs of one call may not overlap, except where a call says
 *     that it works in place.
 *   - Sums, softmax statistics and norms are held in 32 bits or more.  Each
 *     call gives the same bits for the same arguments: no sum goes through
 *     atomics.
 *   - Calls can be captured into a graph: they only launch kernels.
 */
#ifndef ZSMR_OPS_H
#define ZSMR_OPS_H

#include "zsmr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a third format: tensors of a gradient list, matrices, logits */
#define ZSMR_FP32 3

/* Limits of the 2-D operators: rows of at most 2^21 elements (also the
 * strides), at most 2^24 tokens and 2^30 rows of a table. */
#define ZSMR_MAX_WIDTH  ((int64_t)1 << 21)
#define ZSMR_MAX_TOKENS ((int64_t)1 << 24)
#define ZSMR_MAX_VOCAB  ((int64_t)1 << 30)

/* ---- embedding ---------------------------------------------------------
 * ids: n_tokens token ids of id_bytes each (4: int32, 8: int64).  An id
 * outside [0, vocab) is padding: its output row is zero and it has no
 * gradient.  dtype: ZSMR_FP16 or ZSMR_BF16, of the table and of the rows;
 * strides are elements from row to row, at least width. */

/* out[t, :] = RNE16(scale * table[id_t, :]). */
int32_t zsmr_embed_lookup(const void* table, int64_t vocab, int64_t width, int64_t table_stride,
                          int32_t dtype, const void* ids, int32_t id_bytes, int64_t n_tokens,
                          float scale, void* out, int64_t out_stride, hipStream_t stream);

/* Bytes of workspace of zsmr_embed_grad, or -1 for sizes it refuses. */
int64_t zsmr_embed_grad_workspace(int64_t vocab, int64_t width, int64_t n_tokens);

/* dtable[v, :] = RNE16([dtable[v, :] +] scale * sum of dout[t, :] over the
 * tokens with id_t = v).  accumulate == 0: every row is written, those of
 * absent tokens with zeros (a rank's gradient row is read whole by the
 * reduce).  accumulate == 1: the sum is added to what is there and rows of
 * absent tokens stay untouched (an embedding tied to the output head).  The
 * sum is fp32, in an order that depends on the ids alone. */
int32_t zsmr_embed_grad(const void* dout, int64_t dout_stride, int32_t dtype, const void* ids,
                        int32_t id_bytes, int64_t n_tokens, int64_t vocab, int64_t width,
                        float scale, int32_t accumulate, void* dtable, int64_t dtable_stride,
                        void* ws, int64_t ws_bytes, hipStream_t stream);

/* ---- softmax cross entropy of the output head ----------------------------
 * x: the last hidden states, n_tokens x width; w: the head, vocab x width;
 * labels as ids above (outside [0, vocab): the token does not count, its loss
 * and gradient are zero, and its x and weight may hold anything).  With s[t, v] = x[t, :] . w[v, :],
 *   lse[t] = log sum_v exp s[t, v],   loss[t] = lse[t] - s[t, label_t].
 * A logit below -2.3e38 counts as -infinity; one above 2.3e38 makes lse infinite.
 * The logits exist a tile (forward) or a piece of the vocabulary (backward,
 * as 16-bit probabilities) at a time. */

/* Bytes of workspace of a forward call (backward == 0), or of both calls
 * (backward == 1); -1 for sizes they refuse.  It serves operands of any stride
 * and alignment: a copy of x and of up to 32,768 rows of w (268 MB at width
 * 4,096) is part of it, of which w's is left alone where 16-byte loads can read
 * w.  The backward pass's probabilities are the most of it otherwise: 512 MB at
 * most, and 512 bytes a token from 2^20 tokens on. */
int64_t zsmr_xent_workspace(int64_t n_tokens, int64_t vocab, int64_t width, int32_t backward);

/* loss and lse: n_tokens fp32 each (lse of every token, labelled or not).
 * summary: three fp32, {mean loss over the tokens that count, 1 / their
 * number, their number}; all zero if none counts. */
int32_t zsmr_xent_forward(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                          int32_t dtype, const void* labels, int32_t id_bytes, int64_t n_tokens,
                          int64_t vocab, int64_t width, float* loss, float* lse, float* summary,
                          void* ws, int64_t ws_bytes, hipStream_t stream);

/* Gradients of sum_t grad[t] * scale * loss[t]:
 *   G[t, v] = (exp(s[t, v] - lse[t]) - [v == label_t]) * grad[t]
 *   dx = RNE16(scale * G w),   dw = RNE16([dw +] scale * G^T x).
 * lse as the forward call left it.  grad: n_tokens fp32, or NULL for ones;
 * scale: one fp32 on the device, or NULL for 1 (the mean's is summary + 1).
 * dx or dw may be NULL: that gradient is left out.  accumulate == 1 adds to
 * dw.  G is rounded to 16 bits for the matrix instructions that use it.  In
 * fp16 it is held times a power of two that brings the largest |grad| of the
 * tokens that count to 2^14..2^15, one for all tokens: what lies below 2^-28 of
 * that weight is rounded to steps of 2^-39 of it.  So in fp16 the dx row of a
 * token whose weight is 1e-5 or less of the largest has fewer bits than its
 * neighbours'; bf16 has fp32's range and no such limit. */
int32_t zsmr_xent_backward(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                           int32_t dtype, const void* labels, int32_t id_bytes, int64_t n_tokens,
                           int64_t vocab, int64_t width, const float* lse, const float* grad,
                           const float* scale, void* dx, int64_t dx_stride, void* dw,
                           int64_t dw_stride, int32_t accumulate, void* ws, int64_t ws_bytes,
                           hipStream_t stream);

/* ---- global norm and clipping --------------------------------------------
 * A list of n_tensors contiguous tensors: ptrs[i] (device), numels[i] >= 0
 * and dtypes[i] (ZSMR_FP16, ZSMR_BF16 or ZSMR_FP32), host arrays that are
 * read before the call returns. */

/* Bytes of workspace of the calls below for lists of up to n_tensors tensors
 * of up to total elements in all (n_tensors = 1 and total = the piece's
 * length for zero_reduce_shard_sumsq); -1 for sizes they refuse. */
int64_t zsmr_norm_workspace(int64_t total, int32_t n_tensors);

/* norm_coef[0] = the L2 norm of all elements of the list, norm_coef[1] =
 * min(1, max_norm / (norm + eps)); squares and sums in 64 bits, each rounded
 * to fp32 once.  A NaN gives NaN for both, an infinity a coefficient of 0.
 * max_norm and eps: finite, >= 0. */
int32_t zsmr_grad_norm(const void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                       int32_t n_tensors, double max_norm, double eps, float* norm_coef, void* ws,
                       int64_t ws_bytes, hipStream_t stream);

/* The same from n sums of squares (fp64, on the device) of disjoint parts:
 * one of each rank's shard, joined in order as an all-reduce would leave it. */
int32_t zsmr_clip_coef(const double* sums, int64_t n, double max_norm, double eps,
                       float* norm_coef, hipStream_t stream);

/* In place: every element times coef[0] (one fp32 on the device), rounded to
 * its format once.  A coefficient of exactly 1 leaves the tensors unread. */
int32_t zsmr_clip_grads(void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                        int32_t n_tensors, const float* coef, hipStream_t stream);

/* The list, times coef[0] (NULL: 1), concatenated in order into a rank's flat
 * 16-bit gradient row of flat_numel elements; what the list does not fill is
 * zero (the pad of ZeroAdam._flatten).  ZSMR_ERR_ARG if it does not fit. */
int32_t zsmr_clip_flatten(const void* const* ptrs, const int64_t* numels, const int32_t* dtypes,
                          int32_t n_tensors, const float* coef, void* flat, int64_t flat_numel,
                          int32_t flat_dtype, hipStream_t stream);

/* ---- the clipped shard step ----------------------------------------------
 * The global norm depends on every rank's reduced gradient, so the step is two
 * passes with the join between them: zero_reduce_shard_sumsq on every piece,
 * zsmr_clip_coef on the sums, zero_clipped_step on every piece.  A piece has
 * fewer than 2^35 elements, otherwise ZSMR_ERR_ARG. */

/* zero_reduce_shard (the same bits in g_out, the same counting), and in the
 * same pass sumsq[0] = the sum of the squares of g_out (fp64, device). */
int32_t zero_reduce_shard_sumsq(zsmr_ctx* ctx, int32_t rank, int32_t unit, const void* grads,
                                int64_t row_stride, int64_t base_elem, int32_t mean, float* g_out,
                                double* sumsq, void* ws, int64_t ws_bytes, hipStream_t stream);

/* Adam on coef[0] * g (one fp32 rounding; coef NULL: g itself) and the cast
 * of the updated master, in one pass over the (rank, unit) piece.  The bits
 * of zero_adam_step on the multiplied gradient + zero_gather_cast, counted as
 * the latter. */
int32_t zero_clipped_step(zsmr_ctx* ctx, int32_t rank, int32_t unit, const float* g,
                          const float* coef, float* master, float* m, float* v, void* p16_dst,
                          int32_t t, const zsmr_adam* hp, hipStream_t stream);

/* ---- the orthogonalised update --------------------------------------------
 * From X0 = x / (|x|_F + eps), for each of `steps` triples (a, b, c):
 *   X' = a X + (b A + c A^2) X,  A = X X^T  (for a matrix taller than wide: of
 *   its transpose),
 * an odd polynomial that moves every singular value the way the triple says:
 * with a = 3.4445, b = -4.7750, c = 2.0315 five times, to about 1.  Every
 * product has fp32's accuracy (operands of 22 bits, fp32 sums), whatever the
 * formats of x and out.  An operand is no finer than 2^-39 of the largest value that
 * the steps allow its matrix, or of 1: what is that small beside it (an x far below eps,
 * singular values that a step shrinks to nothing) has fewer bits.  For 16-bit results, and in the shard step, steps may share
 * their products with X, which leaves up to three times the error of single steps: of
 * the 2-norm 2e-6 to 6e-6 for white noise (single 1e-6 to 2e-6, products of fp32
 * operands 1e-6 to 5e-6), 2e-4 near rank one (1.7e-4, 2.7e-4).  A matrix of zeros
 * gives zeros; one with a NaN or an infinity gives NaN. */
#define ZSMR_MAX_NS_STEPS 16
typedef struct zsmr_newton {
    double eps;                             /* finite, >= 0 */
    int32_t steps;                          /* 1 .. ZSMR_MAX_NS_STEPS */
    int32_t pad;
    double coef[ZSMR_MAX_NS_STEPS][3];      /* finite; no step may move a singular value beyond 181,
                                             * nor make b s^2 + c s^4 larger than 32,768 */
} zsmr_newton;

/* Sides of a matrix at most 2^18, elements at most 2^33, matrices of a call at
 * most 2^20. */
#define ZSMR_MAX_SIDE     ((int64_t)1 << 18)
#define ZSMR_MAX_MATRIX   ((int64_t)1 << 33)
#define ZSMR_MAX_MATRICES ((int64_t)1 << 20)

/* Bytes of workspace of the two calls below, or -1 for sizes they refuse.  For the
 * matrices that are worked on at a time (2^25 elements at most, or one matrix) 8 bytes
 * an element, and an element of the inner m x m matrix, m the shorter side, 8, or 20
 * where the longer side is 1.2 m or more; rows count with a padding to 32.  Matrices of
 * up to 2^25 elements need less than 1.0 GB, however many there are.  It serves every
 * format of the result and every list of steps, so a call may leave some of it alone. */
int64_t zsmr_orthogonalize_workspace(int64_t rows, int64_t cols, int64_t count);

/* out[k] = the last X of x[k], rounded to out_dtype once, for `count` matrices of
 * rows x cols: x_stride and out_stride elements from row to row (at least cols),
 * x_batch and out_batch from matrix to matrix (any, as long as the matrices of out do
 * not overlap).  out may be x, in the same format and layout, or memory apart from it.
 * Formats: ZSMR_FP16, ZSMR_BF16 or ZSMR_FP32.  The bits of a matrix do not depend on
 * what the others hold, but on how many a call has. */
int32_t zsmr_orthogonalize(const void* x, int32_t x_dtype, int64_t x_stride, int64_t x_batch,
                           void* out, int32_t out_dtype, int64_t out_stride, int64_t out_batch,
                           int64_t rows, int64_t cols, int64_t count, const zsmr_newton* ns,
                           void* ws, int64_t ws_bytes, hipStream_t stream);

/* lr, weight_decay, scale: finite, >= 0, and lr * weight_decay and lr * scale in fp32's
 * range; 0 <= beta < 1; nesterov 0 or 1. */
typedef struct zsmr_muon {
    double lr, beta, weight_decay, scale;
    int32_t nesterov, pad;
} zsmr_muon;

/* The shard step of matrices that a rank holds whole: `count` matrices of rows x
 * cols, row by row and one behind the other, from element `begin` of the (rank,
 * unit) piece on.  With g = mean over the ranks (zero_reduce_shard):
 *   momentum = beta * momentum + g,  u = nesterov ? g + beta * momentum : momentum,
 *   master = (1 - lr * weight_decay) * master - (lr * scale) * orthogonalised(u),
 *   p16 = RNE16(master),
 * every operation outside the products rounded to fp32.  Pointers and base_elem
 * refer to the whole piece, and the call counts as zero_fused_step_range on these
 * elements does.  ZSMR_ERR_ARG if the matrices reach past the piece, and at stage
 * ZSMR_DP unless they are the whole vector.  A rank that holds nothing of the unit
 * has no matrices: ZSMR_ERR_ARG unless count is 0, which does nothing. */
int32_t zero_muon_step(zsmr_ctx* ctx, int32_t rank, int32_t unit, int64_t begin, int64_t rows,
                       int64_t cols, int64_t count, const void* grads, int64_t row_stride,
                       int64_t base_elem, float* master, float* momentum, void* p16_dst,
                       const zsmr_muon* hp, const zsmr_newton* ns, void* ws, int64_t ws_bytes,
                       hipStream_t stream);

/* ---- scores of logits ------------------------------------------------------
 * logits: n_tokens rows of vocab (at most 2^21) elements, ZSMR_FP16, ZSMR_BF16 or
 * ZSMR_FP32, stride elements apart.  With z = scale * logit, in fp32,
 *   lse = log sum_v exp z_v,  logprob = z_id - lse,  p_v = exp(z_v - lse),
 *   entropy = -sum_v p_v log p_v.
 * Logits of -infinity are masked: p = 0.  So are values of z below -2.3e38, which
 * the lowest values of bf16 and fp32 are unless scale makes them larger; that of fp16,
 * -65,504, and other finite masks are ordinary logits.  A row with nothing else has lse
 * -infinity, entropy 0, log probabilities of -infinity and a gradient of zeros.  A
 * NaN makes a row's lse, logprob, entropy and gradient NaN; +infinity, or a z above
 * 2.3e38, makes its lse +infinity and leaves the rest of the row's results but the
 * alternatives' indices unspecified.  An id outside [0, vocab) is
 * padding: logprob 0, which has no gradient; entropy and alternatives are the
 * row's.  scale: 2^-100 .. 2^100. */
#define ZSMR_MAX_TOP 64

/* Bytes of workspace, or -1 for sizes the call refuses. */
int64_t zsmr_logprobs_workspace(int64_t n_tokens, int64_t vocab, int32_t top);

/* logprob, lse, entropy: n_tokens fp32 each; any may be NULL, logprob has to be
 * where ids is.  top (0 .. ZSMR_MAX_TOP, at most vocab): the alternatives of
 * largest logit, the lowest index first among equal ones: n_tokens x top indices of
 * top_bytes each (4 or 8) and their log probabilities in fp32; either may be NULL.
 * Rows with fewer logits above -infinity end in -1 and -infinity; NaN is no
 * alternative. */
int32_t zsmr_logprobs(const void* logits, int64_t stride, int32_t dtype, const void* ids,
                      int32_t id_bytes, int64_t n_tokens, int64_t vocab, float scale,
                      float* logprob, float* lse, float* entropy, int32_t top, void* top_ids,
                      int32_t top_bytes, float* top_logprobs, void* ws, int64_t ws_bytes,
                      hipStream_t stream);

/* dlogits = RNE(scale * (g * ([v = id] - p_v) - h * p_v * (log p_v + entropy))), the
 * gradient of sum (g * logprob + h * entropy), in the format of the logits, whose
 * memory it may share (the same address and stride).  g and h: n_tokens fp32 each, or
 * NULL for zeros; entropy may be NULL where h is, ids where g is.  lse and entropy
 * are what zsmr_logprobs left.  An lse in fp32 holds less of log p the larger it is: a row
 * of |lse| above 512 (fp16), 4,096 (bf16) or 64 (fp32) is summed again from its logits. */
int32_t zsmr_logprobs_grad(const void* logits, int64_t stride, int32_t dtype, const void* ids,
                           int32_t id_bytes, int64_t n_tokens, int64_t vocab, float scale,
                           const float* lse, const float* entropy, const float* g, const float* h,
                           void* dlogits, int64_t dlogits_stride, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* ZSMR_OPS_H */
