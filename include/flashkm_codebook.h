/*
 * flashkm_codebook.h — C ABI of the codebook operators: table lookup with
 * scaling, its gradient by sorted ids, and the balance loss of a router's or
 * codebook's use with its counts and gradient.
 *
 * They stand next to the k-means entry points of flashkm.h: the labels that
 * kmeans_assign / kmeans_assign_top2 write are the ids of kmeans_embed and the
 * selections of kmeans_balance, a table is a centroid array (of any of the
 * three types here), and the gradient uses the same stable inverse mapping of
 * the ids as the centroid update.
 *
 * Conventions as in flashkm.h (status codes, kmeans_last_error, device
 * pointers owned by the caller, contiguous row-major arrays, work only
 * enqueued on `stream`, arguments validated before anything is enqueued,
 * bitwise determinism, nothing allocated), and:
 *   Shapes: B instances (B = 1 is the plain problem) of N rows.  N may be 0
 *     and may be below or above K; pointers to arrays without elements may be
 *     null.  B >= 1, K >= 1, 1 <= D <= 2^20, B*N < 2^31, B*K < 2^31.
 *   Any D and K; pointers need their element type's alignment only (rows of
 *     whole 16-byte words at 16-byte addresses move fastest).
 *   Outputs must not overlap inputs (KM_EINVAL).
 *   NaN and infinities in the data propagate as IEEE arithmetic has it; what
 *     an id outside [0,K) or an invalid row hides is never read into a result.
 *   Calls that share a workspace must be ordered on one stream.
 */
#ifndef FLASHKM_CODEBOOK_H
#define FLASHKM_CODEBOOK_H

#include "flashkm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Lookup with scaling:
 *   out[b,i,:] = round(scale * table[b, ids[b,i], :])   for 0 <= ids[b,i] < K
 *              = 0                                        otherwise (padding)
 * table [B,K,D] table_dtype, ids [B,N] int32, out [B,N,D] out_dtype.  The
 * product is fp32, rounded once (to nearest even) into out_dtype. */
KM_API int kmeans_embed(const void* table, int32_t table_dtype, int64_t N, int32_t K, int32_t D, int32_t B,
                        const int32_t* ids, float scale, void* out, int32_t out_dtype, void* stream);

/* Bytes of device workspace kmeans_embed_grad needs for this shape (0 for an
 * invalid shape; 256 where none is needed: `ws` may then be null; the same for
 * every type). */
KM_API size_t kmeans_embed_grad_workspace_bytes(int64_t N, int32_t K, int32_t D, int32_t B);

/* Gradient of the lookup with respect to the table:
 *   grad[b,k,:] = (accumulate ? grad[b,k,:] : 0)
 *                 + scale * sum over i with ids[b,i] = k of dout[b,i,:]
 * dout [B,N,D] dout_dtype, ids [B,N] int32 (rows with ids outside [0,K) leave
 * nothing), grad [B,K,D] grad_dtype.  Sums are fp32 in a fixed order of the
 * id-sorted rows, scaled and (when accumulating) added to the old value in
 * fp32, then rounded once into grad_dtype.  With `accumulate` an entry that no
 * row names is left as it is, bit for bit; without it such an entry is 0. */
KM_API int kmeans_embed_grad(const void* dout, int32_t dout_dtype, int64_t N, int32_t K, int32_t D, int32_t B,
                             const int32_t* ids, float scale, int32_t accumulate, void* grad, int32_t grad_dtype,
                             void* ws, size_t ws_bytes, void* stream);

/* Bytes of device workspace kmeans_balance needs for this shape (0 for an
 * invalid shape; 256 where none is needed: `ws` may then be null; the same for
 * every type). */
KM_API size_t kmeans_balance_workspace_bytes(int64_t N, int32_t K, int32_t B, int32_t S);

/* Balance loss of the use of K choices by N rows, with counts:
 *   p[b,i,:]    = softmax(logits[b,i,:])
 *   lse[b,i]    = log sum_k exp(logits[b,i,k])        (+inf for an invalid row)
 *   T           = valid rows of instance b
 *   prob[b,k]   = (1/T) sum over valid i of p[b,i,k]
 *   counts[b,k] = #{(i,s) : i valid, labels[b,i,s] = k}
 *   loss[b]     = K * sum_k counts[b,k] / (S T) * prob[b,k]
 *   coef[b,k]   = K * counts[b,k] / (S T^2), the derivative of loss[b] with
 *                 respect to each valid row's p[b,i,k]
 * logits [B,N,K] dtype, labels [B,N,S] int32 (1 <= S, B*N*S < 2^31; a label
 * outside [0,K) names nothing but stays in the S T that counts are divided
 * by), valid [B,N] bytes (nullable: every row; non-zero = valid); loss [B]
 * fp32, counts [B,K] int32, prob [B,K] fp32, lse [B,N] fp32, coef [B,K] fp32.
 * At most 2^22 instances.
 * T = 0 gives loss, prob and coef 0.  A valid row whose logits are all -inf
 * has lse -inf and leaves no probability (it still counts in T).  A choice with
 * logit -inf has probability 0.  A valid row with a NaN or a +inf has no
 * softmax (inf - inf): its lse is NaN, never the +inf of an invalid row, and
 * prob and loss of its instance are NaN; counts, coef and the other rows' lse
 * are not touched by it.  Balanced use gives loss 1. */
KM_API int kmeans_balance(const void* logits, int32_t dtype, int64_t N, int32_t K, int32_t B,
                          const int32_t* labels, int32_t S, const uint8_t* valid, float* loss, int32_t* counts,
                          float* prob, float* lse, float* coef, void* ws, size_t ws_bytes, void* stream);

/* Gradient of the balance loss with respect to the logits, from the lse and
 * coef of kmeans_balance and the derivative dloss [B] fp32 of what follows:
 *   p              = softmax(logits[b,i,:])
 *   dlogits[b,i,:] = dloss[b] * p * (coef[b,:] - sum_k p_k coef[b,k])
 * rounded once into dtype.  lse says which rows have probabilities: rows with
 * lse +inf (invalid) or -inf (nothing left) get zeros, whatever their logits
 * hold; a row with lse NaN gets NaN.  For the others it is only the shift of the
 * exponentials, whose sum is taken from the logits again (an fp32 lse of large
 * magnitude does not hold the logarithm of the sum): a value near the row's log
 * sum exp gives the same p, one far from it overflows or leaves nothing. */
KM_API int kmeans_balance_grad(const void* logits, int32_t dtype, int64_t N, int32_t K, int32_t B,
                               const float* lse, const float* coef, const float* dloss, void* dlogits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASHKM_CODEBOOK_H */
