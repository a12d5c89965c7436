/*
 * qlora_logprobs.h -- log probabilities of given tokens, with entropy and
 * the best alternatives, and the gradient of the logits.
 *
 * For each row of logits x (V values), with m = max_j x_j,
 * l = log sum_j exp(x_j - m), logp_j = (x_j - m) - l and p_j = exp(logp_j):
 *
 *     logprob = logp_t                    (t the row's target)
 *     entropy = -sum_j p_j logp_j
 *     top     the n largest logits, by value descending, then index ascending
 *
 * What training reads off the head's output (the token loss is the mean of
 * -logprob; preference and policy losses weigh logprob and entropy) and what
 * serving returns beside a token. The conventions of qlora_nf4.h hold.
 * Everything is computed in float32 from logits of bf16 or float32.
 *
 * Special rows
 *   - A logit of -inf (a banned token) has p = 0 and adds nothing.
 *   - A row of -inf only: max -inf, l 0, every logp -inf, entropy 0, its
 *     gradient 0.
 *   - A row holding +inf or NaN: logprob, entropy, the alternatives' log
 *     probabilities and its gradient are NaN (NaN ranks above +inf).
 *   - A target outside [0, V) (an ignored position, e.g. -100): logprob 0
 *     and no gradient from it; entropy and alternatives as for any row.
 */
#ifndef QLORA_LOGPROBS_H
#define QLORA_LOGPROBS_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QLORA_DTYPE_BF16 = 0, QLORA_DTYPE_F32 = 1 };

#define QLORA_MAX_TOP 32

/*
 * Logits: N rows of V values, row i at data + i * ld elements (ld >= V).
 * `data` is 16-byte aligned (else QLORA_ERR_INVALID_ARG); ld is any number of
 * elements, so that the other rows start at any element.
 */
typedef struct qlora_logits {
  void *data;
  int64_t N, V, ld;
  int32_t dtype;           /* QLORA_DTYPE_* */
  int32_t reserved;        /* set to 0 */
} qlora_logits;

/* Workspace in bytes (0: none needed); (size_t)-1 for an unsupported shape. */
QLORA_API size_t qlora_token_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t dtype,
                                                      int32_t top);

/*
 * targets [N] int64; logprob [N]; stats [N][2] = (m, l), which the gradient
 * needs; entropy [N] or NULL; top_logprobs [N][top] float32 and top_ids
 * [N][top] int64 for 0 <= top <= min(V, QLORA_MAX_TOP) (NULL when top is 0).
 * N < 1, V < 1, ld < V, top < 0 or top > V: QLORA_ERR_INVALID_ARG. V >= 2^31 - 2^16,
 * N >= 2^31, ld > 2^40, top > QLORA_MAX_TOP (and <= V), or a shape too large for one
 * launch (2^32 threads: more than about 16 million short rows): QLORA_ERR_UNSUPPORTED.
 * The gradient's shapes have the same limits. targets and top_ids are 8-byte, the
 * float outputs 4-byte aligned.
 */
QLORA_API qlora_status qlora_token_logprobs(const qlora_logits *logits, const int64_t *targets,
                                            float *logprob, float *stats, float *entropy,
                                            int32_t top, float *top_logprobs, int64_t *top_ids,
                                            void *ws, size_t ws_bytes, void *stream);

/*
 * Gradient of the logits for upstream gradients dlogprob [N] and, unless
 * NULL, dentropy [N] (entropy then as the forward wrote it):
 *   dx_j = dlogprob (delta_jt - p_j) - dentropy p_j (logp_j + entropy)
 * into dlogits (the same N, V and dtype; any ld >= V; elements past V are
 * left as they are). dlogits->data may be logits->data with the same ld (the
 * logits are then replaced by their gradient), otherwise they must not
 * overlap. A row whose target is ignored or whose dlogprob is 0, and whose
 * dentropy is 0 or absent, gets zeros whatever it holds.
 */
QLORA_API qlora_status qlora_token_logprobs_bwd(const qlora_logits *logits, const int64_t *targets,
                                                const float *stats, const float *entropy,
                                                const float *dlogprob, const float *dentropy,
                                                const qlora_logits *dlogits, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_LOGPROBS_H */
