// Log probabilities of given tokens with entropy and the best alternatives,
// and the gradient of the logits, gfx950 (include/qlora_logprobs.h).
//
// With m = max_j x_j, t_j = x_j - m, z = sum exp(t_j) and l = log z:
//   logprob = t_target - l,   entropy = l - (sum exp(t_j) t_j) / z,
//   dx_j = g (delta - p_j) - e p_j (logp_j + entropy),  logp_j = t_j - l.
// Differences from the maximum keep every quantity near zero where the
// logits themselves are large. Sums are float32.
#include "../../include/qlora_logprobs.h"
#include "capi_util.h"

namespace {

constexpr int LT = 256;

struct LpArgs {
  const void *x;
  int64_t N, V, ld;
  const int64_t *targets;
  float *logprob, *stats, *entropy;
  int top;
  float *top_lp;
  int64_t *top_ids;
};

template <bool F32>
QL_DEV float load1(const void *row, int64_t j) {
  return F32 ? ((const float *)row)[j] : ql::bf16_to_f(((const uint16_t *)row)[j]);
}
template <bool F32>
QL_DEV const void *row_of(const void *x, int64_t i, int64_t ld) {
  return (const char *)x + i * ld * (F32 ? 4 : 2);
}

// Order of the alternatives as one integer: value (NaN above +inf, the two
// zeros equal) in the upper half, complement of the index in the lower.
QL_DEV uint64_t order_key(float v, uint32_t j) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = v != v ? 0xff800001u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return ((uint64_t)k << 32) | (0xffffffffu - j);
}

template <class T, class Op>
QL_DEV T block_reduce(T v, T *tmp, Op op) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = op(v, __shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  v = tmp[0];
#pragma unroll
  for (int w = 1; w < LT / 64; ++w) v = op(v, tmp[w]);
  return v;
}

// One workgroup per row: a pass for the maximum, one for the sums, one per
// alternative.
template <bool F32>
__global__ __launch_bounds__(LT) void logprobs_kernel(LpArgs g) {
  __shared__ float tf[LT / 64];
  __shared__ uint64_t tk[LT / 64];
  const int64_t i = blockIdx.x;
  const void *row = row_of<F32>(g.x, i, g.ld);
  const int tid = threadIdx.x;
  float m = -INFINITY;
  for (int64_t j = tid; j < g.V; j += LT) m = fmaxf(m, load1<F32>(row, j));
  m = block_reduce(m, tf, [](float a, float b) { return fmaxf(a, b); });
  const float mm = m == -INFINITY ? 0.0f : m;
  float z = 0.0f, s = 0.0f;
  for (int64_t j = tid; j < g.V; j += LT) {
    const float t = load1<F32>(row, j) - mm;
    const float e = expf(t);
    z += e;
    s += e * fmaxf(t, -1e30f);
  }
  z = block_reduce(z, tf, [](float a, float b) { return a + b; });
  s = block_reduce(s, tf, [](float a, float b) { return a + b; });
  const bool empty = z == 0.0f;          // every logit -inf
  const float l = empty ? 0.0f : logf(z);
  if (tid == 0) {
    const int64_t t = g.targets[i];
    float lp = 0.0f;
    if (t >= 0 && t < g.V) lp = empty ? -INFINITY : (load1<F32>(row, t) - mm) - l;
    g.logprob[i] = lp;
    g.stats[2 * i] = m;
    g.stats[2 * i + 1] = l;
    if (g.entropy) g.entropy[i] = empty ? 0.0f : l - s / z;
  }
  uint64_t last = ~0ull;
  for (int q = 0; q < g.top; ++q) {
    uint64_t best = 0;
    for (int64_t j = tid; j < g.V; j += LT) {
      const uint64_t k = order_key(load1<F32>(row, j), (uint32_t)j);
      if (k < last && k > best) best = k;
    }
    last = block_reduce(best, tk, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    if (tid == 0) {
      const int64_t j = 0xffffffffu - (uint32_t)last;
      g.top_ids[i * g.top + q] = j;
      g.top_lp[i * g.top + q] = empty ? -INFINITY : (load1<F32>(row, j) - mm) - l;
    }
  }
}

struct LpGradArgs {
  const void *x;
  int64_t N, V, ld, ldo;
  const int64_t *targets;
  const float *stats, *entropy, *dlp, *dent;
  void *dx;
};

template <bool F32>
__global__ __launch_bounds__(LT) void logprobs_grad_kernel(LpGradArgs g) {
  const int64_t i = blockIdx.x;
  const void *row = row_of<F32>(g.x, i, g.ld);
  char *out = (char *)g.dx + i * g.ldo * (F32 ? 4 : 2);
  const int64_t t = g.targets[i];
  const float gl = (t >= 0 && t < g.V) ? g.dlp[i] : 0.0f;
  const float ge = g.dent ? g.dent[i] : 0.0f;
  const float ent = g.dent ? g.entropy[i] : 0.0f;
  const float m = g.stats[2 * i], l = g.stats[2 * i + 1];
  const bool zero = (gl == 0.0f && ge == 0.0f) || (m == -INFINITY && l == 0.0f);
  for (int64_t j = threadIdx.x; j < g.V; j += LT) {
    float d = 0.0f;
    if (!zero) {
      const float lp = (load1<F32>(row, j) - m) - l;
      const float p = expf(lp);
      d = -p * (gl + ge * (fmaxf(lp, -1e30f) + ent)) + (j == t ? gl : 0.0f);
    }
    if (F32)
      ((float *)out)[j] = d;
    else
      ((uint16_t *)out)[j] = ql::f_to_bf16(d);
  }
}

constexpr int64_t kMaxV = (int64_t(1) << 31) - (1 << 16);

qlora_status check_logits(const qlora_logits *x) {
  if (!x || x->N < 1 || x->V < 1 || x->ld < x->V || !x->data || !aligned16(x->data))
    return QLORA_ERR_INVALID_ARG;
  if (x->dtype != QLORA_DTYPE_BF16 && x->dtype != QLORA_DTYPE_F32) return QLORA_ERR_INVALID_ARG;
  if (x->V >= kMaxV || x->N > 0x7fffffff || x->ld > (int64_t(1) << 40))
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool aligned8(const void *p) { return ((uintptr_t)p & 7u) == 0; }

}  // namespace

extern "C" {

size_t qlora_token_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t dtype, int32_t top) {
  if (N < 1 || V < 1 || V >= kMaxV || N > 0x7fffffff || top < 0 || top > QLORA_MAX_TOP ||
      top > V || (dtype != QLORA_DTYPE_BF16 && dtype != QLORA_DTYPE_F32))
    return (size_t)-1;
  return 0;
}

qlora_status qlora_token_logprobs(const qlora_logits *x, const int64_t *targets, float *logprob,
                                  float *stats, float *entropy, int32_t top, float *top_logprobs,
                                  int64_t *top_ids, void *ws, size_t ws_bytes, void *stream) {
  qlora_status s = check_logits(x);
  if (s != QLORA_OK) return s;
  if (!targets || !logprob || !stats || !aligned8(targets) || !aligned4(logprob) ||
      !aligned4(stats) || !aligned4(entropy) || top < 0 || top > x->V)
    return QLORA_ERR_INVALID_ARG;
  if (top > QLORA_MAX_TOP) return QLORA_ERR_UNSUPPORTED;
  if (top && (!top_logprobs || !top_ids || !aligned4(top_logprobs) || !aligned8(top_ids)))
    return QLORA_ERR_INVALID_ARG;
  const size_t need = qlora_token_logprobs_workspace_bytes(x->N, x->V, x->dtype, top);
  if (!ws_ok(ws, ws_bytes, (int64_t)need)) return QLORA_ERR_WORKSPACE;
  const LpArgs g{x->data, x->N, x->V, x->ld, targets, logprob, stats, entropy, top, top_logprobs,
                 top_ids};
  hipStream_t st = (hipStream_t)stream;
  QlProf prof(QLORA_K_LOGPROBS, st);
  if (x->dtype == QLORA_DTYPE_F32)
    logprobs_kernel<true><<<(unsigned)x->N, LT, 0, st>>>(g);
  else
    logprobs_kernel<false><<<(unsigned)x->N, LT, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

qlora_status qlora_token_logprobs_bwd(const qlora_logits *x, const int64_t *targets,
                                      const float *stats, const float *entropy,
                                      const float *dlogprob, const float *dentropy,
                                      const qlora_logits *dx, void *stream) {
  qlora_status s;
  if ((s = check_logits(x)) != QLORA_OK || (s = check_logits(dx)) != QLORA_OK) return s;
  if (dx->N != x->N || dx->V != x->V || dx->dtype != x->dtype) return QLORA_ERR_INVALID_ARG;
  if (dx->data == x->data && dx->ld != x->ld) return QLORA_ERR_INVALID_ARG;
  if (!targets || !stats || !dlogprob || !aligned8(targets) || !aligned4(stats) ||
      !aligned4(dlogprob) || !aligned4(dentropy) || !aligned4(entropy))
    return QLORA_ERR_INVALID_ARG;
  if (dentropy && !entropy) return QLORA_ERR_INVALID_ARG;
  const LpGradArgs g{x->data, x->N,    x->V,     x->ld,    dx->ld,  targets,
                     stats,   entropy, dlogprob, dentropy, dx->data};
  hipStream_t st = (hipStream_t)stream;
  QlProf prof(QLORA_K_LOGPROBS_GRAD, st);
  if (x->dtype == QLORA_DTYPE_F32)
    logprobs_grad_kernel<true><<<(unsigned)x->N, LT, 0, st>>>(g);
  else
    logprobs_grad_kernel<false><<<(unsigned)x->N, LT, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

}  // extern "C"
