// C ABI of the orthogonalised momentum step (include/qlora_muon.h): argument
// checks and dispatch.
#include "../../include/qlora_muon.h"
#include "capi_util.h"

namespace {

// Grid limits: matrices are a grid's second dimension; a matrix's chunks of
// the long side are indexed in 32 bits.
bool muon_shape_ok(int64_t n, int64_t rows, int64_t cols) {
  const int64_t small = rows < cols ? rows : cols, len = rows < cols ? cols : rows;
  return n <= 65535 && small <= QLORA_MUON_MAX_RANK && len <= (int64_t(1) << 24);
}
// S is carried by S' = P S P, apart from u. A direction of a small singular value
// has an eigenvalue of S that is wrong by about 2^-53 of the largest, and below
// zero as often as above: every step multiplies it by a^2, and one that comes
// near -1 would run to infinity, as all of P's terms then add up. The update's
// error is 0.1 to 0.6 of a^(2 steps) 2^-53 of its largest direction over spectra
// of eight decades. At the limit, 2^-17 (10 steps of the usual coefficients, 30 of
// 1.5 and -0.5), that is spread over a matrix of 16 x 4096 and times lr = 0.02 less
// than the rounding of its float32 parameters. One step does not use S'.
bool steps_ok(double a, int steps) {
  return steps <= 1 || fabs(a) <= 1.0 || 2.0 * steps * log2(fabs(a)) <= 36.0;
}
bool not_negative(double x) { return isfinite((float)x) && x >= 0.0; }

}  // namespace

extern "C" {

size_t qlora_muon_workspace_bytes(int64_t n, int64_t rows, int64_t cols) {
  if (n < 1 || rows < 1 || cols < 1 || !muon_shape_ok(n, rows, cols)) return (size_t)-1;
  return muon_ws_bytes(n, rows, cols);
}

qlora_status qlora_muon_step(float *param, float *momentum, const uint16_t *grad,
                             uint16_t *param_bf16, int64_t n, int64_t rows, int64_t cols,
                             const qlora_muon_hparams *hp, void *ws, size_t ws_bytes,
                             void *stream) {
  if (!param || !momentum || !grad || !param_bf16 || !hp || n < 1 || rows < 1 || cols < 1)
    return QLORA_ERR_INVALID_ARG;
  if (!muon_shape_ok(n, rows, cols)) return QLORA_ERR_UNSUPPORTED;
  if (!aligned16(param) || !aligned16(momentum) || !aligned16(grad) || !aligned16(param_bf16))
    return QLORA_ERR_INVALID_ARG;
  if (!not_negative(hp->lr) || !not_negative(hp->weight_decay) || !not_negative(hp->eps) ||
      !(hp->beta >= 0.0 && hp->beta < 1.0) || !isfinite((float)hp->scale) || !isfinite(hp->a) ||
      !isfinite(hp->b) || !isfinite(hp->c))
    return QLORA_ERR_INVALID_ARG;
  if (hp->steps < 0 || hp->steps > QLORA_MUON_MAX_STEPS || (hp->nesterov & ~1))
    return QLORA_ERR_INVALID_ARG;
  if (!steps_ok(hp->a, hp->steps)) return QLORA_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, (int64_t)muon_ws_bytes(n, rows, cols))) return QLORA_ERR_WORKSPACE;
  void *dv[4];
  const void *hv[4] = {param, momentum, grad, param_bf16};
  for (int i = 0; i < 4; ++i)
    if (!device_view(hv[i], &dv[i])) return QLORA_ERR_INVALID_ARG;
  const MuonScalars s{(float)hp->beta, (float)(1.0 - hp->beta), (float)hp->lr, (float)hp->scale,
                      (float)hp->weight_decay, hp->eps, hp->a, hp->b, hp->c, hp->steps,
                      hp->nesterov};
  return launch_muon((float *)dv[0], (float *)dv[1], (const uint16_t *)dv[2], (uint16_t *)dv[3], n,
                     rows, cols, s, ws, (hipStream_t)stream);
}

}  // extern "C"
