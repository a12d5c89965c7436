// Argument checks and workspace carving shared by the C-ABI files. Every
// check runs on the host before anything is enqueued.
#pragma once

#include <math.h>

#include "kernels.h"

namespace {

constexpr int64_t kAlign = 256;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Shape checks shared by all entry points.
qlora_status check_weight_shape(int64_t d, int64_t k) {
  if (d < 1 || k < 1) return QLORA_ERR_INVALID_ARG;
  if (k % 64 != 0 || d % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  if (d > (int64_t(1) << 31) || k > (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED;
  const int64_t n = d * k;
  if (n / 64 >= (int64_t(1) << 32)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

qlora_status check_weight(const qlora_nf4_weight *w, bool need_outputs_only) {
  (void)need_outputs_only;
  if (!w) return QLORA_ERR_INVALID_ARG;
  qlora_status s = check_weight_shape(w->d, w->k);
  if (s != QLORA_OK) return s;
  if (w->blocksize != 64) return QLORA_ERR_UNSUPPORTED;
  if (w->double_quant != 0 && w->double_quant != 1) return QLORA_ERR_INVALID_ARG;
  if (w->double_quant && w->dq_blocksize != 256) return QLORA_ERR_UNSUPPORTED;
  if (!w->codes || !aligned16(w->codes)) return QLORA_ERR_INVALID_ARG;
  if (w->double_quant) {
    if (!w->absmax_q || !w->absmax_scale || !w->absmax_offset) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(w->absmax_q)) return QLORA_ERR_INVALID_ARG;  // read as dwords
    if (((uintptr_t)w->absmax_scale & 3u) || ((uintptr_t)w->absmax_offset & 3u))
      return QLORA_ERR_INVALID_ARG;
  } else {
    if (!w->absmax || ((uintptr_t)w->absmax & 3u)) return QLORA_ERR_INVALID_ARG;
  }
  return QLORA_OK;
}

ql::ScaleSrc scale_src(const qlora_nf4_weight *w) {
  return ql::ScaleSrc{w->absmax, w->absmax_q, w->absmax_scale, w->absmax_offset,
                      w->double_quant};
}

// Bump allocator over the caller's workspace (also used to size it).
struct Carve {
  char *base;
  int64_t off = 0;
  template <class T>
  T *take(int64_t bytes) {
    T *p = base ? (T *)(base + off) : nullptr;
    off += ql_rup(bytes > 0 ? bytes : 0, kAlign);
    return p;
  }
};

bool ws_ok(const void *ws, size_t ws_bytes, int64_t need) {
  if (need == 0) return true;
  return ws && (((uintptr_t)ws & (kAlign - 1)) == 0) && (int64_t)ws_bytes >= need;
}

}  // namespace
