/*
 * qlora_adapters.h -- many LoRA adapters on one frozen NF4 base weight.
 *
 * The layer of qlora_nf4.h for a batch whose tokens belong to different
 * adapters (many requests served, or many adapters trained, on one resident
 * base): token m uses adapter a = ids[m], or none,
 *
 *     Y[m]  = X[m] W'^T + s_a (X[m] A_a^T) B_a^T          (none: X[m] W'^T)
 *     dX[m] = dY[m] W'  + s_a (dY[m] B_a) A_a             (none: dY[m] W')
 *     dA_a  = s_a sum_{m: a(m)=a} (dY[m] B_a)^T X[m]
 *     dB_a  = s_a sum_{m: a(m)=a} dY[m]^T (X[m] A_a^T)
 *
 * The base weight is read once for the whole batch. The conventions of
 * qlora_nf4.h hold (device pointers owned by the caller and 16-byte aligned,
 * work only enqueued on `stream`, host checks before anything is enqueued,
 * outputs do not alias inputs, bit-identical results on every call), and one
 * more: the values of a token depend on its own row and its own adapter
 * only. An infinity or NaN in another token's row or another adapter's
 * matrices does not reach it, and among batches of the same M a token's H, Y
 * and dX are a function, bit for bit, of its row, its adapter and the adapter's
 * number, wherever the token stands and whatever the others use. Batches of
 * other sizes may add in another order.
 */
#ifndef QLORA_ADAPTERS_H
#define QLORA_ADAPTERS_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest adapter count of one call, most tokens of one plan, and most tokens
 * of one linear (a launch of more threads than a grid holds otherwise). */
#define QLORA_MAX_ADAPTERS 1024
#define QLORA_MAX_PLAN_TOKENS ((int64_t)1 << 30)
#define QLORA_MAX_ADAPTER_TOKENS ((int64_t)1 << 24)

/*
 * The adapters of one linear: n adapters of r ranks each.
 *   A      [n][r][k] bf16;  B [n][d][r] bf16
 *   scale  [n] float32: s_a (alpha_a over the adapter's own rank)
 * An adapter of fewer ranks is stored with zero rows of A and zero columns
 * of B. 1 <= n <= QLORA_MAX_ADAPTERS (more: QLORA_ERR_UNSUPPORTED),
 * 1 <= r <= 128 (as in qlora_nf4.h).
 */
typedef struct qlora_adapters {
  int32_t n;
  int32_t r;
  const uint16_t *A;
  const uint16_t *B;
  const float *scale;      /* 4-byte aligned */
} qlora_adapters;

/*
 * Which tokens use which adapter: built once per batch on the device
 * (qlora_adapter_plan_build) and used by every linear the batch passes. `data` is
 * device memory of qlora_adapter_plan_bytes(M, n) bytes, owned by the
 * caller; it must hold a plan built for the same M and n before (in stream
 * order) the calls that take it, which only read it.
 */
typedef struct qlora_adapter_plan {
  int64_t M;               /* tokens */
  int32_t n;               /* adapters */
  int32_t reserved;        /* set to 0 */
  void *data;
  size_t bytes;
} qlora_adapter_plan;

/* Bytes of a plan; 0 for M < 1, M > QLORA_MAX_PLAN_TOKENS, n < 1 or
 * n > QLORA_MAX_ADAPTERS. */
QLORA_API size_t qlora_adapter_plan_bytes(int64_t M, int32_t n);

/*
 * Build the plan of ids [M] (int32, 4-byte aligned). Any id outside [0, n)
 * means no adapter. Tokens are ordered by adapter, tokens of one adapter in
 * batch order. One launch. M or n below 1 return QLORA_ERR_INVALID_ARG, above
 * their limits QLORA_ERR_UNSUPPORTED, and `bytes` too small
 * QLORA_ERR_WORKSPACE; the calls that take a plan check it the same way.
 */
QLORA_API qlora_status qlora_adapter_plan_build(const int32_t *ids, const qlora_adapter_plan *plan,
                                                void *stream);

/* Device workspace of the calls below in bytes for op QLORA_OP_FWD or
 * QLORA_OP_BWD; (size_t)-1 for an unsupported shape (M above
 * QLORA_MAX_ADAPTER_TOKENS is one, QLORA_ERR_UNSUPPORTED in the calls). */
QLORA_API size_t qlora_adapters_workspace_bytes(int32_t op, int64_t d, int64_t k, int64_t M,
                                                int32_t n, int32_t r);

/*
 * Forward: Y (M x d, bf16), X M x k bf16, M = plan->M. If H_save is
 * non-NULL it receives H[m] = X[m] A_a^T (M x r float32; zero rows for
 * tokens without an adapter) for the backward pass. M <= 16 runs the
 * memory-bound decode kernels, larger M the fused dequant-GEMM; both read
 * each touched adapter's matrices in place. As in qlora_linear_fwd, W'
 * enters the matrix units as bf16: the GEMM (and every backward) as w' =
 * bf16(level a'), the decode kernels as bf16(level), times a' in float32
 * after each block's sum; the two differ by the rounding of a weight. Adapter-input dropout (the
 * qlora_dropout of qlora_nf4.h) is not offered here.
 */
QLORA_API qlora_status qlora_linear_fwd_adapters(const qlora_nf4_weight *w, const uint16_t *X,
                                                 const qlora_adapters *adapters,
                                                 const qlora_adapter_plan *plan, uint16_t *Y,
                                                 float *H_save, void *ws, size_t ws_bytes,
                                                 void *stream);

/*
 * Backward of the forward above for dY (M x d, bf16): dX (M x k; skipped when
 * NULL), dA [n][r][k] and dB [n][d][r] (bf16, every entry written; zero for
 * adapters without tokens). H is the forward's H_save (M x r float32), or
 * NULL to recompute it.
 */
QLORA_API qlora_status qlora_linear_bwd_adapters(const qlora_nf4_weight *w, const uint16_t *X,
                                                 const qlora_adapters *adapters,
                                                 const qlora_adapter_plan *plan,
                                                 const uint16_t *dY, const float *H, uint16_t *dX,
                                                 uint16_t *dA, uint16_t *dB, void *ws,
                                                 size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_ADAPTERS_H */
