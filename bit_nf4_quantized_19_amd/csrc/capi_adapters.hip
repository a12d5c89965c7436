// C ABI of the many-adapter linear (include/qlora_adapters.h): argument
// checks, workspace layout and dispatch.
#include "../../include/qlora_adapters.h"
#include "capi_util.h"

namespace {

bool plan_shape_ok(int64_t M, int32_t n) {
  return M >= 1 && M <= QLORA_MAX_PLAN_TOKENS && n >= 1 && n <= QLORA_MAX_ADAPTERS;
}

qlora_status check_plan(const qlora_adapter_plan *p) {
  if (!p || p->M < 1 || p->n < 1) return QLORA_ERR_INVALID_ARG;
  if (!plan_shape_ok(p->M, p->n)) return QLORA_ERR_UNSUPPORTED;
  if (!p->data || !aligned16(p->data)) return QLORA_ERR_INVALID_ARG;
  if (p->bytes < AdapterPlan(nullptr, p->M, p->n).bytes) return QLORA_ERR_WORKSPACE;
  return QLORA_OK;
}

qlora_status check_adapters(const qlora_adapters *a, const qlora_adapter_plan *p) {
  if (!a || a->n < 1 || a->r < 1) return QLORA_ERR_INVALID_ARG;
  if (a->n > QLORA_MAX_ADAPTERS || a->r > 128) return QLORA_ERR_UNSUPPORTED;
  if (!a->A || !a->B || !aligned16(a->A) || !aligned16(a->B)) return QLORA_ERR_INVALID_ARG;
  if (!a->scale || ((uintptr_t)a->scale & 3u)) return QLORA_ERR_INVALID_ARG;
  return a->n == p->n ? QLORA_OK : QLORA_ERR_INVALID_ARG;
}

struct FwdWs {
  uint16_t *hi, *lo;   // M > 16: s_a H in plan order
  float *part;         // partial sums: M <= 16 of slices and H, larger M of split tiles
  int64_t bytes;
};
FwdWs fwd_layout(char *base, int64_t d, int64_t k, int64_t M, int r) {
  const int rp = (int)ql_rup(r, 16);
  Carve c{base};
  FwdWs L{};
  if (M > 16) {
    L.hi = c.take<uint16_t>(M * rp * 2);
    L.lo = c.take<uint16_t>(M * rp * 2);
    L.part = c.take<float>((int64_t)gemm_adapter_part_bytes(M, d, k));
  } else {
    L.part = c.take<float>((int64_t)gemv_part_bytes(d, k, M, rp, 1));
  }
  L.bytes = c.off;
  return L;
}

struct BwdWs {
  float *H, *G;
  float *part;         // partial sums of the gradients, then of dX's split tiles
  uint16_t *hi, *lo;
  int *ctr;            // counters of the gradients
  int64_t bytes;
};
BwdWs bwd_layout(char *base, int64_t d, int64_t k, const AdapterPlan &plan, int r) {
  const int rp = (int)ql_rup(r, 16);
  Carve c{base};
  BwdWs L{};
  L.H = c.take<float>(plan.M * r * 4);
  L.G = c.take<float>(plan.M * rp * 4);
  L.hi = c.take<uint16_t>(plan.M * rp * 2);
  L.lo = c.take<uint16_t>(plan.M * rp * 2);
  L.ctr = c.take<int>(4 * colacc_adapters_counter_count(plan, d, k));
  const size_t pg = colacc_adapters_part_bytes(plan, d, k, rp);
  const size_t px = gemm_adapter_part_bytes(plan.M, k, d);
  L.part = c.take<float>((int64_t)(pg > px ? pg : px));
  L.bytes = c.off;
  return L;
}

}  // namespace

extern "C" {

size_t qlora_adapter_plan_bytes(int64_t M, int32_t n) {
  return plan_shape_ok(M, n) ? AdapterPlan(nullptr, M, n).bytes : 0;
}

qlora_status qlora_adapter_plan_build(const int32_t *ids, const qlora_adapter_plan *plan,
                                      void *stream) {
  const qlora_status s = check_plan(plan);
  if (s != QLORA_OK) return s;
  if (!ids || ((uintptr_t)ids & 3u)) return QLORA_ERR_INVALID_ARG;
  return launch_adapter_plan(ids, AdapterPlan(plan->data, plan->M, plan->n),
                             (hipStream_t)stream);
}

size_t qlora_adapters_workspace_bytes(int32_t op, int64_t d, int64_t k, int64_t M, int32_t n,
                                      int32_t r) {
  if (check_weight_shape(d, k) != QLORA_OK || !plan_shape_ok(M, n) ||
      M > QLORA_MAX_ADAPTER_TOKENS || r < 1 || r > 128)
    return (size_t)-1;
  if (op == QLORA_OP_FWD) return (size_t)fwd_layout(nullptr, d, k, M, r).bytes;
  if (op == QLORA_OP_BWD)
    return (size_t)bwd_layout(nullptr, d, k, AdapterPlan(nullptr, M, n), r).bytes;
  return (size_t)-1;
}

qlora_status qlora_linear_fwd_adapters(const qlora_nf4_weight *w, const uint16_t *X,
                                       const qlora_adapters *ad, const qlora_adapter_plan *plan,
                                       uint16_t *Y, float *H_save, void *ws, size_t ws_bytes,
                                       void *stream) {
  qlora_status s;
  if ((s = check_weight(w, false)) != QLORA_OK || (s = check_plan(plan)) != QLORA_OK ||
      (s = check_adapters(ad, plan)) != QLORA_OK)
    return s;
  if (!X || !Y || !aligned16(X) || !aligned16(Y) || !aligned16(H_save))
    return QLORA_ERR_INVALID_ARG;
  const int64_t d = w->d, k = w->k, M = plan->M;
  if (M > QLORA_MAX_ADAPTER_TOKENS) return QLORA_ERR_UNSUPPORTED;
  const int r = ad->r, rp = (int)ql_rup(r, 16);
  const FwdWs L = fwd_layout((char *)ws, d, k, M, r);
  if (!ws_ok(ws, ws_bytes, L.bytes)) return QLORA_ERR_WORKSPACE;
  const AdapterPlan p(plan->data, M, plan->n);
  hipStream_t st = (hipStream_t)stream;
  if (M <= 16) {
    const GemvIn in{w->codes, scale_src(w), d, ad->A, ad->B, H_save, Y,
                    DropParams{0u, 0u, 0u, 1.0f, 0}};
    return launch_gemv_adapters(in, k, X, M, r, rp, p.tok, p.n, ad->scale, L.part, st);
  }
  if ((s = launch_skinny_adapters(X, k, ad->A, ad->scale, p, false, r, rp, nullptr, H_save, L.hi,
                                  L.lo, st)) != QLORA_OK)
    return s;
  const GemmAdapters ga{p.perm, p.sid, L.part};
  return launch_gemm_fwd(w->codes, scale_src(w), d, k, X, M, ad->B, r, L.hi, L.lo, rp, Y, st, &ga);
}

qlora_status qlora_linear_bwd_adapters(const qlora_nf4_weight *w, const uint16_t *X,
                                       const qlora_adapters *ad, const qlora_adapter_plan *plan,
                                       const uint16_t *dY, const float *H, uint16_t *dX,
                                       uint16_t *dA, uint16_t *dB, void *ws, size_t ws_bytes,
                                       void *stream) {
  qlora_status s;
  if ((s = check_weight(w, false)) != QLORA_OK || (s = check_plan(plan)) != QLORA_OK ||
      (s = check_adapters(ad, plan)) != QLORA_OK)
    return s;
  if (!X || !dY || !dA || !dB || !aligned16(X) || !aligned16(dY) || !aligned16(dA) ||
      !aligned16(dB) || !aligned16(dX) || !aligned16(H))
    return QLORA_ERR_INVALID_ARG;
  const int64_t d = w->d, k = w->k, M = plan->M;
  if (M > QLORA_MAX_ADAPTER_TOKENS) return QLORA_ERR_UNSUPPORTED;
  const int r = ad->r, rp = (int)ql_rup(r, 16);
  const AdapterPlan p(plan->data, M, plan->n);
  const BwdWs L = bwd_layout((char *)ws, d, k, p, r);
  if (!ws_ok(ws, ws_bytes, L.bytes)) return QLORA_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  if (!H) {
    if ((s = launch_skinny_adapters(X, k, ad->A, ad->scale, p, false, r, rp, nullptr, L.H, nullptr,
                                    nullptr, st)) != QLORA_OK)
      return s;
    H = L.H;
  }
  // G = dY B_a, which also clears the counters of the gradient launch
  if ((s = launch_skinny_adapters(dY, d, ad->B, ad->scale, p, true, r, rp, L.G, nullptr, L.hi,
                                  L.lo, st, L.ctr, colacc_adapters_counter_count(p, d, k))) !=
      QLORA_OK)
    return s;
  // dB_a = s_a dY^T H and dA_a = s_a G^T X over each adapter's tokens
  if ((s = launch_colacc2_adapters(ColaccAdReq{dY, d, H, r, dB, 0},
                                   ColaccAdReq{X, k, L.G, rp, dA, 1}, p, rp, r, ad->scale, L.part,
                                   L.ctr, st)) != QLORA_OK)
    return s;
  if (!dX) return QLORA_OK;
  const GemmAdapters ga{p.perm, p.sid, L.part};
  return launch_gemm_dx(w->codes, scale_src(w), d, k, dY, M, ad->A, r, L.hi, L.lo, rp, dX, nullptr,
                        1.0f, st, &ga);
}

}  // extern "C"
