// C ABI of the 8-bit base (include/qlora_int8.h): argument checks, workspace
// layout and dispatch.
#include "../../include/qlora_int8.h"
#include "capi_util.h"

namespace {

qlora_status check_shape(int64_t d, int64_t k) {
  const qlora_status s = check_weight_shape(d, k);
  if (s != QLORA_OK) return s;
  return d <= QLORA_INT8_MAX_DIM && k <= QLORA_INT8_MAX_DIM ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}

qlora_status check_record(const qlora_int8_weight *w) {
  if (!w) return QLORA_ERR_INVALID_ARG;
  const qlora_status s = check_shape(w->d, w->k);
  if (s != QLORA_OK) return s;
  if (!w->codes || !w->scale || !aligned16(w->codes) || !aligned16(w->scale))
    return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

// r == 0: no adapter, and none of the adapter's arrays
qlora_status check_rank(int32_t r, float alpha, bool any, bool all) {
  if (r < 0) return QLORA_ERR_INVALID_ARG;
  if (r > 128) return QLORA_ERR_UNSUPPORTED;
  if (r == 0) return any ? QLORA_ERR_INVALID_ARG : QLORA_OK;
  return all && isfinite(alpha) ? QLORA_OK : QLORA_ERR_INVALID_ARG;
}

struct FwdWs {
  int8_t *q;           // M x ldq codes of the tokens
  float *sx;
  float *H;            // M x rp
  uint16_t *hi, *lo;   // s H
  void *part;
  int64_t ldq, bytes;
};
// any: sized for every call of up to M tokens, whose partial sums may be larger
FwdWs fwd_layout(char *base, int64_t d, int64_t k, int64_t M, int r, bool any = false) {
  const int64_t rp = ql_rup(r, 16);
  Carve c{base};
  FwdWs L{};
  L.ldq = ql_rup(k, 128);
  L.q = c.take<int8_t>(M * L.ldq);
  L.sx = c.take<float>(M * 4);
  L.H = c.take<float>(M * rp * 4);
  L.hi = c.take<uint16_t>(M * rp * 2);
  L.lo = c.take<uint16_t>(M * rp * 2);
  L.part = c.take<void>(M <= INT8_GEMV_TOKENS ? 0
                        : (int64_t)(any ? int8_gemm_part_bytes_upto(M, d, k)
                                        : int8_gemm_part_bytes(M, d, k)));
  L.bytes = c.off;
  return L;
}

struct BwdWs {
  int8_t *q;           // M x ldq codes of dY sw
  float *se, *H, *G, *cpart;
  void *part;
  uint16_t *At, *Bt, *hi, *lo;
  int64_t ldq, bytes;
};
// sized for the largest case (H recomputed, dX requested)
BwdWs bwd_layout(char *base, int64_t d, int64_t k, int64_t M, int r, bool any = false) {
  const int rp = (int)ql_rup(r, 16);
  Carve c{base};
  BwdWs L{};
  L.ldq = ql_rup(d, 128);
  L.q = c.take<int8_t>(M * L.ldq);
  L.se = c.take<float>(M * 4);
  if (r) {
    L.H = c.take<float>(M * rp * 4);
    L.G = c.take<float>(M * rp * 4);
    L.hi = c.take<uint16_t>(M * rp * 2);
    L.lo = c.take<uint16_t>(M * rp * 2);
    L.At = c.take<uint16_t>((int64_t)rp * k * 2);
    L.Bt = c.take<uint16_t>((int64_t)rp * d * 2);
    L.cpart = c.take<float>((int64_t)colacc_part_bytes(M, d, k, rp));
  }
  L.part = c.take<void>((int64_t)(any ? int8_gemm_part_bytes_upto(M, k, d)
                                      : int8_gemm_part_bytes(M, k, d)));
  L.bytes = c.off;
  return L;
}

}  // namespace

extern "C" {

qlora_status qlora_int8_quantize(const uint16_t *W, const qlora_int8_weight *out, void *stream) {
  const qlora_status s = check_record(out);
  if (s != QLORA_OK) return s;
  if (!W || !aligned16(W)) return QLORA_ERR_INVALID_ARG;
  return launch_int8_rows(W, out->d, out->k, nullptr, out->codes, out->k, out->scale,
                          (hipStream_t)stream);
}

size_t qlora_int8_workspace_bytes(int32_t op, int64_t d, int64_t k, int64_t M, int32_t r) {
  if (check_shape(d, k) != QLORA_OK || M < 1 || M > QLORA_INT8_MAX_TOKENS || r < 0 || r > 128)
    return (size_t)-1;
  if (op == QLORA_OP_FWD) return (size_t)fwd_layout(nullptr, d, k, M, r, true).bytes;
  if (op == QLORA_OP_BWD) return (size_t)bwd_layout(nullptr, d, k, M, r, true).bytes;
  return (size_t)-1;
}

qlora_status qlora_linear_fwd_int8(const qlora_int8_weight *w, const uint16_t *X, int64_t M,
                                   const uint16_t *A, const uint16_t *B, int32_t r,
                                   float lora_alpha, uint16_t *Y, float *H_save, void *ws,
                                   size_t ws_bytes, void *stream) {
  qlora_status s;
  if ((s = check_record(w)) != QLORA_OK ||
      (s = check_rank(r, lora_alpha, A || B || H_save, A && B)) != QLORA_OK)
    return s;
  if (!X || !Y || M < 1 || !aligned16(X) || !aligned16(Y) || !aligned16(A) || !aligned16(B) ||
      !aligned16(H_save))
    return QLORA_ERR_INVALID_ARG;
  if (M > QLORA_INT8_MAX_TOKENS) return QLORA_ERR_UNSUPPORTED;
  const int64_t d = w->d, k = w->k;
  const FwdWs L = fwd_layout((char *)ws, d, k, M, r);
  if (!ws_ok(ws, ws_bytes, L.bytes)) return QLORA_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  const int rp = (int)ql_rup(r, 16);
  const float sc = r ? lora_alpha / (float)r : 0.0f;
  const Int8Rank rank{A, r, r, rp, L.H, H_save, L.hi, L.lo, sc, nullptr, 0};
  s = r ? launch_int8_prep(X, M, k, nullptr, L.q, L.ldq, L.sx, rank, st)
        : launch_int8_rows(X, M, k, nullptr, L.q, L.ldq, L.sx, st);
  if (s != QLORA_OK) return s;
  if (M <= INT8_GEMV_TOKENS)
    return launch_int8_gemv(w->codes, w->scale, d, k, L.q, L.ldq, L.sx, M, B, L.hi, L.lo, r, rp, Y,
                            st);
  return launch_int8_gemm(0, w->codes, w->scale, d, k, L.q, L.ldq, L.sx, M, B, r, L.hi, L.lo, rp,
                          Y, L.part, st);
}

qlora_status qlora_linear_bwd_int8(const qlora_int8_weight *w, const uint16_t *X, int64_t M,
                                   const uint16_t *A, const uint16_t *B, int32_t r,
                                   float lora_alpha, const uint16_t *dY, const float *H,
                                   uint16_t *dX, uint16_t *dA, uint16_t *dB, void *ws,
                                   size_t ws_bytes, void *stream) {
  qlora_status s;
  if ((s = check_record(w)) != QLORA_OK ||
      (s = check_rank(r, lora_alpha, A || B || H || dA || dB, A && B && dA && dB && X)) !=
          QLORA_OK)
    return s;
  if (!dY || M < 1 || (r == 0 && !dX)) return QLORA_ERR_INVALID_ARG;
  for (const void *p : {(const void *)X, (const void *)A, (const void *)B, (const void *)dY,
                        (const void *)H, (const void *)dX, (const void *)dA, (const void *)dB})
    if (!aligned16(p)) return QLORA_ERR_INVALID_ARG;
  if (M > QLORA_INT8_MAX_TOKENS) return QLORA_ERR_UNSUPPORTED;
  const int64_t d = w->d, k = w->k;
  const BwdWs L = bwd_layout((char *)ws, d, k, M, r);
  if (!ws_ok(ws, ws_bytes, L.bytes)) return QLORA_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  const int rp = (int)ql_rup(r, 16);
  const float sc = r ? lora_alpha / (float)r : 0.0f;
  if (r) {
    // B^T for G and A^T for dX, which are read by rows, and H as M x rp
    const float *pad = r % 16 ? H : nullptr;
    if ((s = launch_int8_layout(A, B, d, k, r, rp, L.At, L.Bt, pad, M, L.H, st)) != QLORA_OK)
      return s;
    if (pad) {
      H = L.H;
    } else if (!H) {
      const Int8Rank rank{A, r, r, rp, L.H, nullptr, nullptr, nullptr, sc, nullptr, 0};
      if ((s = launch_int8_prep(X, M, k, nullptr, nullptr, 0, nullptr, rank, st)) != QLORA_OK)
        return s;
      H = L.H;
    }
    // G = dY B, s G as bf16 hi/lo and the record of dY sw; the launch also
    // clears the counters of the gradients' launch
    const Int8Rank rank{L.Bt, rp, r, rp, L.G, nullptr, L.hi, L.lo, sc,
                        colacc_counters(L.cpart, M, d, k, rp), colacc_counter_count(d, k)};
    if ((s = launch_int8_prep(dY, M, d, w->scale, dX ? L.q : nullptr, L.ldq, L.se, rank, st)) !=
        QLORA_OK)
      return s;
    const DropParams none{0u, 0u, 0u, 1.0f, 0};
    if ((s = launch_colacc2(ColaccReq{dY, d, H, dB, 0, none, nullptr},
                            ColaccReq{X, k, L.G, dA, 1, none, nullptr}, M, rp, r, sc, L.cpart,
                            st)) != QLORA_OK)
      return s;
  }
  if (!dX) return QLORA_OK;
  if (!r && (s = launch_int8_rows(dY, M, d, w->scale, L.q, L.ldq, L.se, st)) != QLORA_OK) return s;
  return launch_int8_gemm(1, w->codes, w->scale, d, k, L.q, L.ldq, L.se, M, L.At, rp, L.hi, L.lo,
                          rp, dX, L.part, st);
}

}  // extern "C"
