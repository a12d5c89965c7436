/*
 * qlora_int8.h -- a frozen 8-bit integer base weight with a LoRA branch.
 *
 * The linear layer of qlora_nf4.h on a base stored as one int8 code per weight
 * and one float32 scale per output channel (row), multiplied with the tokens
 * in integers. A record of rows x cols bf16 values is, per row i,
 *
 *     s_i  = fl32(max_j |w_ij| / 127)
 *     q_ij = min(max(rne(fl32(w_ij / s_i)), -127), 127)     (s_i = 0: q_ij = 0)
 *
 * (fl32: correctly rounded float32, rne: nearest whole number, ties to even).
 * With (Xq, sx) the record of the tokens X (M x k) and (Wq, sw) that of the
 * weight (d x k), s = lora_alpha / r, A (r x k) and B (d x r):
 *
 *     Y  = sx sw (Xq Wq^T) + s H B^T,   H = X A^T
 *     dX = se (Eq Wq) + s G A,          G = dY B
 *     dA = s G^T X,                     dB = s dY^T H
 *
 * where (Eq, se) is the record of the rows of fl32(dY sw): the channel scales
 * lie along the contraction of dX, so they are folded in before a token's
 * codes are taken. The rounding of X is passed straight through by the
 * backward, and that of dY sw changes an entry by at most se / 2. The sums of
 * code products are exact (int32), so they do not depend on how a call is
 * split; the LoRA branch reads X and dY unquantised. H and G are float32 sums;
 * s H and s G enter Y and dX, and H and G enter dB and dA, as two bf16 parts
 * that leave out at most 2^-16 of each value (an output is rounded to bf16, 2^-8
 * of its own), with products and sums in float32.
 *
 * Conventions of qlora_nf4.h: every array is caller-owned device memory,
 * 16-byte aligned unless stated, every call only enqueues work on `stream`,
 * validates on the host before anything is enqueued and allocates nothing;
 * outputs do not alias inputs; repeated calls give identical bits. A token's
 * values depend on its own row only: a NaN or an infinity in a row of X (dY)
 * makes that row of Y (dX) NaN and reaches no other. A row of a weight that
 * holds one makes that column of Y NaN, and dX whole.
 */
#ifndef QLORA_INT8_H
#define QLORA_INT8_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest contraction whose int32 sum cannot overflow (127^2 * 131072 < 2^31),
 * hence largest d and k, and most tokens of one call. */
#define QLORA_INT8_MAX_DIM ((int64_t)131072)
#define QLORA_INT8_MAX_TOKENS ((int64_t)1 << 20)

/*
 * The 8-bit base weight. d % 8 == 0, k % 64 == 0, both at most
 * QLORA_INT8_MAX_DIM (otherwise QLORA_ERR_UNSUPPORTED).
 */
typedef struct qlora_int8_weight {
  int64_t d, k;
  int8_t *codes;           /* [d][k] */
  float *scale;            /* [d] */
} qlora_int8_weight;

/*
 * The record of a bf16 matrix W (d x k, row-major): writes out->codes and
 * out->scale. One launch. Also the record of any matrix of such rows.
 */
QLORA_API qlora_status qlora_int8_quantize(const uint16_t *W, const qlora_int8_weight *out,
                                           void *stream);

/* Device workspace of the calls below in bytes for op QLORA_OP_FWD or
 * QLORA_OP_BWD, up to M tokens and up to rank r (0: no adapter); (size_t)-1 for
 * an unsupported shape. */
QLORA_API size_t qlora_int8_workspace_bytes(int32_t op, int64_t d, int64_t k, int64_t M,
                                            int32_t r);

/*
 * Forward: Y (M x d, bf16) of X (M x k, bf16). 1 <= r <= 128, or r == 0 with A,
 * B and H_save NULL for the product alone (a merged weight). If H_save is
 * non-NULL it receives H (M x r float32) for the backward. Up to 16 tokens
 * run the memory-bound decode kernel, more the integer GEMM.
 */
QLORA_API qlora_status qlora_linear_fwd_int8(const qlora_int8_weight *w, const uint16_t *X,
                                             int64_t M, const uint16_t *A, const uint16_t *B,
                                             int32_t r, float lora_alpha, uint16_t *Y,
                                             float *H_save, void *ws, size_t ws_bytes,
                                             void *stream);

/*
 * Backward for dY (M x d, bf16): dX (M x k; skipped when NULL), dA (r x k) and
 * dB (d x r), bf16. H is the forward's H_save, or NULL to recompute it. With
 * r == 0 only dX is computed: A, B, H, dA and dB are NULL, dX is not, and X is
 * not read (may be NULL).
 */
QLORA_API qlora_status qlora_linear_bwd_int8(const qlora_int8_weight *w, const uint16_t *X,
                                             int64_t M, const uint16_t *A, const uint16_t *B,
                                             int32_t r, float lora_alpha, const uint16_t *dY,
                                             const float *H, uint16_t *dX, uint16_t *dA,
                                             uint16_t *dB, void *ws, size_t ws_bytes,
                                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_INT8_H */
