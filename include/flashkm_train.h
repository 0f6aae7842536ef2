/*
 * flashkm_train.h — C ABI of a training step's other operators: routing of
 * rows to choices (scores, a bias for balance, groups, top-k, weights) with
 * its gradient, and the AdamW step over many tensors with states in 32 bits
 * or in 8.
 *
 * They stand next to the codebook operators of flashkm_codebook.h: the ids
 * that kmeans_route writes are the labels of kmeans_balance (for which -1
 * names nothing) and the ids of kmeans_embed (for which -1 is padding), its
 * gradient can be added onto kmeans_balance_grad's, and the tables whose
 * gradient kmeans_embed_grad writes are stepped by kmeans_adamw.
 *
 * Conventions as in flashkm_codebook.h (status codes, kmeans_last_error,
 * device pointers owned by the caller, contiguous row-major arrays, element
 * alignment, outputs overlap nothing, work only enqueued on `stream`,
 * arguments validated before anything is enqueued, bitwise determinism,
 * nothing allocated).  No call needs a workspace.
 */
#ifndef FLASHKM_TRAIN_H
#define FLASHKM_TRAIN_H

#include "flashkm_codebook.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a row's logits become scores. */
enum km_score { KM_SOFTMAX = 0, KM_SIGMOID = 1 };

/* The most selections a row and the most groups. */
#define KM_ROUTE_MAX_S 64
#define KM_ROUTE_MAX_GROUPS 64

/* Routing of N rows to S of K choices each:
 *   s[i,:] = softmax(logits[i,:]) or sigmoid(logits[i,:])
 *   c[i,k] = s[i,k] + bias[k]; a choice whose logit or c is -inf is out
 *   groups > 1: choices are `groups` groups of K / groups neighbours.  A
 *     group's worth is the sum of its group_best (1 or 2) largest c, of those
 *     that are not out.  The top_groups groups of the largest worth stay (ties
 *     to the lowest index), the other groups' choices are out
 *   ids[i,0..S)  the S choices of the largest c in descending order, ties to
 *     the lowest index; -1 in the last places if fewer are not out
 *   chosen[i,j]  the logit of ids[i,j] in fp32 (-inf for an id of -1)
 *   weights[i,j] scale * s[i,ids[i,j]], or with `renormalise`
 *     scale * s[i,ids[i,j]] / sum over j of s[i,ids[i,j]]; 0 for an id of -1.
 *     The share is formed relative to the largest chosen score, so that scores
 *     too small for fp32 still have one
 * logits [N,K] dtype, bias [K] fp32 (nullable), valid [N] bytes (nullable:
 * every row; non-zero = valid; a row that is not has no choices), ids [N,S]
 * int32, weights [N,S] fp32, chosen [N,S] fp32.  N >= 0, N < 2^31, K >= 1,
 * 1 <= S <= min(K, 64), groups <= 64 divides K, 1 <= top_groups <= groups.
 * Exactness of the ids: where c's order is the logits' own (no bias, and no
 * sums of two c as worths) it is taken from the logits, exactly.  Else it is
 * the order of c and of the worths in 64-bit arithmetic: rows in which 32 bits
 * could change it are decided in 64.  Values that differ by less than the
 * rounding of 64-bit arithmetic (sums of equal parts in another order) come in
 * the order that this rounding gives them.
 * A valid row with a NaN among its logits or the bias, or with a logit of +inf
 * under softmax, has no scores: its ids are -1, its weights and chosen NaN. */
KM_API int kmeans_route(const void* logits, int32_t dtype, int64_t N, int32_t K, const float* bias, int32_t score,
                        int32_t groups, int32_t top_groups, int32_t group_best, int32_t S, int32_t renormalise,
                        float scale, const uint8_t* valid, int32_t* ids, float* weights, float* chosen, void* stream);

/* Gradient of the weights with respect to the logits, the ids held fixed:
 *   dlogits[i,:] = (accumulate ? dlogits[i,:] : 0)
 *                  + d sum_j dweights[i,j] * weights[i,j] / d logits[i,:]
 * with ids and chosen of kmeans_route, dweights [N,S] fp32 the derivative of
 * what follows.  Sums are fp32, rounded once into dtype.  logits [N,K] is read
 * only by softmax without renormalise (which reaches every choice of the row)
 * and may be null otherwise; chosen is read only where logits is not, and may
 * be null there.  An id outside [0,K) leaves nothing, whatever chosen and
 * dweights hold in its place, and a row without another id gets nothing at
 * all.  The same id twice in a row adds up.  With `accumulate` an entry that
 * the row's gradient does not reach is left as it is, bit for bit. */
KM_API int kmeans_route_grad(const void* logits, int32_t dtype, int64_t N, int32_t K, const int32_t* ids,
                             const float* chosen, const float* dweights, int32_t S, int32_t score, int32_t renormalise,
                             float scale, int32_t accumulate, void* dlogits, void* stream);

/* One tensor of an AdamW step: device pointers and the number of elements (0
 * is nothing).  master: an fp32 copy of the parameter that the step is taken
 * on, or null.  States in 32 bits: exp_avg and exp_avg_sq fp32, the scales
 * null.  States in 8 bits: exp_avg e4m3 (OCP, finite and NaN), exp_avg_sq e5m2
 * bytes, and an fp32 scale for each 256 consecutive elements of each.
 * decay multiplies the call's weight_decay for this tensor. */
typedef struct km_adamw_tensor {
  void* param;
  const void* grad;
  float* master;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  int64_t numel;
  float decay;
} km_adamw_tensor;

/* The elements that share a scale. */
#define KM_ADAMW_BLOCK 256

/* Bytes of the table that kmeans_adamw reads for these tensors (host array;
 * only numel is looked at); 0 for invalid arguments. */
KM_API size_t kmeans_adamw_table_bytes(const km_adamw_tensor* tensors, int32_t count);

/* Validates the tensors (1 <= count <= 2^20, all of one parameter type and one
 * gradient type, with a master copy each or none) and writes the table of the
 * step into the HOST memory `table`.  The caller copies it to the device, where
 * it must be 256-byte aligned, and keeps it as long as the tensors stay where
 * they are.  Arrays that a step writes may overlap nothing, in any tensor;
 * gradients may be shared. */
KM_API int kmeans_adamw_table(const km_adamw_tensor* tensors, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                              int32_t bits, void* table, size_t table_bytes);

/* Added to bits = 8 in kmeans_adamw: codes are rounded stochastically. */
#define KM_ADAMW_STOCHASTIC 256

/* One AdamW step over the tensors of a table, in one launch:
 *   g = grad_scale * grad
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * p is the master copy where there is one, and the parameter its value rounded
 * once to param_dtype; arithmetic is fp32 (eps is rounded to it); 0 / 0 (eps 0,
 * nothing moved) is 0.  count, chunks, param_dtype, grad_dtype, bits and
 * masters (0 or 1) are those the table was made for.
 * States in 8 bits: a block's scale is its largest magnitude times 2^-8 (m) or
 * 2^-15 (v; 2^-133 at least), a value is its code times the scale, rounded to
 * nearest even, so the largest is held exactly; a positive v is at least the
 * smallest code (2^-16) and stays positive, so that an element whose v is not
 * 0 in fp32 never divides by eps alone; an m in a block whose largest magnitude
 * is below 2^-100 is held as 0.  The step itself uses m and v before they are
 * rounded.  A NaN stays with its element; an infinite m is held as NaN, an
 * infinite v (the square of a large gradient) as infinity, which stops its
 * element.
 * What nearest rounding means for a run: a code moves only if a step moves its
 * value by half a code, 6 to 12 % for v and 3 to 6 % for m.  beta2 = 0.999 moves
 * v by 0.1 % of its distance from g^2, so a g^2 of about 100 v and more shows
 * and one below does not: an element's v stays where it is relative to its
 * block's largest, which alone follows the average.  Elements whose gradients
 * fall behind their block's take steps that are too small (by 4 to 10 times
 * after some thousand steps), those of a block with one spike steps that are too
 * large.
 * With bits 8 | KM_ADAMW_STOCHASTIC (the table is that of 8) m's and v's codes
 * are rounded stochastically: to one of the two codes next to the value, to
 * either with the probability that makes the expectation the value itself (to
 * 2^-19 of their distance).  What is held then follows the averages without
 * bias, with an error of its own: with beta2 = 0.999 and steady gradients v is
 * off by 33 % at one standard deviation (a step by 17 %), m by 7 % of its size.
 * This is the one to train with for more than some hundred steps.  A block's
 * largest is held exactly and a positive v is at least the smallest code, as
 * above.  The random numbers are a function of the step's number and the
 * element's place in the table, so a run repeats bit for bit, and every step
 * needs a number of its own.
 * Step count and rates that change between replays of a captured call are read
 * on the device: step_at (int64 >= 1, nullable) in place of step, lr_at (fp32,
 * nullable) in place of lr.  grad_scale_at (fp32, nullable) is grad_scale (1
 * if null); skip_at (a byte, nullable): nothing is changed where it is not 0. */
KM_API int kmeans_adamw(const void* table, int32_t count, int64_t chunks, int32_t param_dtype, int32_t grad_dtype,
                        int32_t bits, int32_t masters, double lr, double beta1, double beta2, double eps,
                        double weight_decay, int64_t step, const float* lr_at, const int64_t* step_at,
                        const float* grad_scale_at, const uint8_t* skip_at, void* stream);

/* The chunks of a table: its workgroups, as kmeans_adamw takes them. */
KM_API int64_t kmeans_adamw_chunks(const km_adamw_tensor* tensors, int32_t count);

#ifdef __cplusplus
}
#endif

#endif /* FLASHKM_TRAIN_H */
