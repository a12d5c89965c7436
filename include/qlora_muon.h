/*
 * qlora_muon.h -- orthogonalised momentum step of the LoRA matrices.
 *
 * Beside the AdamW step of qlora_nf4.h: one step on n matrices of the same
 * shape rows x cols (the A or B of one projection over the layers, or one
 * matrix), each on its own:
 *
 *     m' = beta m + (1 - beta) g
 *     u  = (1 - beta) g + beta m'   (nesterov)   or   m'
 *     X0 = u / (|u|_F + eps)
 *     X_{j+1} = (a I + b S + c S^2) X_j,  S = X_j X_j^T,  j = 0 .. steps - 1
 *     p' = p - lr (scale X_steps + weight_decay p),   out = bf16(p')
 *
 * (S on the smaller side; the quintic Newton-Schulz iteration, which moves
 * every singular value of u towards one with the default coefficients). Every
 * factor is a polynomial in the first S, so X_steps = Q X0 with Q a small
 * matrix: u is read twice whatever the number of steps. S and Q are held in
 * float64, m, p and the update in float32, each elementwise operation rounded
 * once in the order written. The rounding of the first S grows by a^2 a step:
 * X_steps is off by less than a^(2 steps) 2^-53 of its largest singular value
 * (with a = 3.4445 2^-35 after 5 steps, 2^-17 after 10), and counts above
 * a^(2 steps) = 2^36 are refused.
 */
#ifndef QLORA_MUON_H
#define QLORA_MUON_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest smaller side of a matrix (the largest rank of an adapter) and most
 * iterations, whatever the coefficients. */
#define QLORA_MUON_MAX_RANK 128
#define QLORA_MUON_MAX_STEPS 32

typedef struct qlora_muon_hparams {
  double lr, beta, weight_decay, eps;
  double scale;            /* of the orthogonalised update */
  double a, b, c;          /* coefficients of an iteration */
  int32_t steps;           /* 0 .. QLORA_MUON_MAX_STEPS (0: u / (|u|_F + eps) itself);
                            * more than one: a^(2 steps) <= 2^36, otherwise
                            * QLORA_ERR_UNSUPPORTED (3.4445: 10 steps, 2: 18, 1.5: 30) */
  int32_t nesterov;        /* 0 or 1 */
} qlora_muon_hparams;

/* Device workspace in bytes of up to n matrices, each with its smaller and its
 * larger side no larger than these; (size_t)-1 for an unsupported shape (n, rows
 * or cols below 1, min(rows, cols) above QLORA_MUON_MAX_RANK, n above 65535 or
 * max(rows, cols) above 2^24). */
QLORA_API size_t qlora_muon_workspace_bytes(int64_t n, int64_t rows, int64_t cols);

/*
 * One step. param, momentum ([n][rows][cols] float32) are updated in place,
 * grad is bf16, param_bf16 receives the bf16 copy of the updated parameters;
 * 16-byte aligned. As in qlora_adamw_step, param and momentum may be device
 * memory or page-locked host memory (paged out); grad, param_bf16 and ws are
 * device memory. Hyperparameters: lr, weight_decay and eps finite and not
 * negative, 0 <= beta < 1, scale, a, b and c finite. A matrix whose update is
 * zero takes the decay alone when eps > 0. A NaN or an infinity in one
 * matrix reaches no other. Only enqueues on `stream`; repeated calls on the
 * same inputs give identical bits.
 */
QLORA_API qlora_status qlora_muon_step(float *param, float *momentum, const uint16_t *grad,
                                       uint16_t *param_bf16, int64_t n, int64_t rows,
                                       int64_t cols, const qlora_muon_hparams *hp, void *ws,
                                       size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_MUON_H */
