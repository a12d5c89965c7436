// Log probabilities of given tokens with entropy and the best alternatives,
// and the gradient of the logits, gfx950 (include/qlora_logprobs.h).
//
// With m = max_j x_j, t_j = x_j - m, z = sum exp(t_j) and l = log z:
//   logprob = t_target - l,   entropy = l - (sum exp(t_j) t_j) / z,
//   dx_j = g (delta - p_j) - e p_j (logp_j + entropy),  logp_j = t_j - l.
// Differences from the maximum keep every quantity near zero where the
// logits themselves are large. Sums are float32.
#include <float.h>

#include <algorithm>

#include "../../include/qlora_logprobs.h"
#include "capi_util.h"

namespace {

constexpr int JT = 256;   // threads of the join and gradient kernels

struct LpArgs {
  const void *x;
  int64_t N, V, ld;
  const int64_t *targets;
  float *logprob, *stats, *entropy;
  int top;
  float *top_lp;
  int64_t *top_ids;
  int64_t chunk;       // logits of a row per workgroup, a multiple of 8
  int nchunk;
  float4 *part;        // [N][nchunk]: m, z, sum exp(t) t of a chunk (nchunk > 1)
  uint64_t *keys;      // [N][nchunk][top]: its best, in order; 0 past its end
};

template <bool F32>
QL_DEV float load1(const void *row, int64_t j) {
  return F32 ? ((const float *)row)[j] : ql::bf16_to_f(((const uint16_t *)row)[j]);
}
template <bool F32>
QL_DEV const void *row_of(const void *x, int64_t i, int64_t ld) {
  return (const char *)x + i * ld * (F32 ? 4 : 2);
}

// 16 bytes of a row: 4 float32 or 8 bf16. Rows start at any element, so the
// accesses are declared with the element's alignment only (the hardware takes
// them at any).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
template <bool F32> constexpr int lp_elems() { return F32 ? 4 : 8; }
template <bool F32>
QL_DEV u32x4 load16(const void *row, int64_t j) {
  if (F32) return *(const u32x4_a4 *)((const float *)row + j);
  return *(const u32x4_a2 *)((const uint16_t *)row + j);
}
template <bool F32>
QL_DEV float elem(const u32x4 &v, int e) {
  if (F32) return __uint_as_float(v[e]);
  return (e & 1) ? ql::bf16hi(v[e >> 1]) : ql::bf16lo(v[e >> 1]);
}

// Order of the alternatives as one integer: value (NaN above +inf, the two
// zeros equal) in the upper half, complement of the index in the lower. Never
// 0 (what is past the end) nor all ones.
QL_DEV uint64_t order_key(float v, uint32_t j) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = v != v ? 0xff800001u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return ((uint64_t)k << 32) | (0xffffffffu - j);
}
QL_DEV float key_value(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

QL_DEV float fast_exp(float t) { return __builtin_amdgcn_exp2f(t * 1.44269504088896340736f); }

struct OpMax {
  template <class T> QL_DEV T operator()(T a, T b) const { return a > b ? a : b; }
  QL_DEV float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <int LT, class T, class Op>
QL_DEV T block_reduce(T v, T *tmp, Op op) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = op(v, (T)__shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  v = tmp[0];
#pragma unroll
  for (int w = 1; w < LT / 64; ++w) v = op(v, tmp[w]);
  return v;
}

// The row's results from its sums (one thread).
template <bool F32>
QL_DEV void finish_row(const LpArgs &g, int64_t i, const void *row, float m, float l, float z,
                       float s, bool empty) {
  const int64_t t = g.targets[i];
  float lp = 0.0f;
  if (t >= 0 && t < g.V)
    lp = empty ? -INFINITY : (load1<F32>(row, t) - m) - l;
  g.logprob[i] = lp;
  g.stats[2 * i] = m;
  g.stats[2 * i + 1] = l;
  if (g.entropy) g.entropy[i] = empty ? 0.0f : l - s / z;
}
QL_DEV void put_top(const LpArgs &g, int64_t i, int q, uint64_t key, float m, float l,
                    bool empty) {
  g.top_ids[i * g.top + q] = (int64_t)(0xffffffffu - (uint32_t)key);
  g.top_lp[i * g.top + q] = empty ? -INFINITY : (key_value(key) - m) - l;
}

// The `top` largest of `count` distinct keys in LDS, by counting the larger
// ones of each; emit(q, key) in order.
template <int LT, class Emit>
QL_DEV void emit_ranked(const uint64_t *list, int count, int top, Emit emit) {
  for (int c = threadIdx.x; c < count; c += LT) {
    const uint64_t k = list[c];
    int rank = 0;
    for (int o = 0; o < count; ++o) rank += list[o] > k ? 1 : 0;
    if (rank < top) emit(rank, k);
  }
}

constexpr int LP_LIST = 1024;   // candidates of a chunk held in LDS
constexpr int LP_GROUPS = 64;   // groups of threads whose maxima give the threshold

// Maximum, sum of exp(x - m) and of exp(x - m)(x - m) over some logits. m
// starts at the lowest finite number, so that differences from it are never
// NaN for want of a logit; z is 0 exactly when every logit is -inf.
struct Sums {
  float m, z, s;
};
QL_DEV Sums sums_at(const Sums &a, float m) {   // a referred to a maximum m >= a.m
  const float d = a.m - m, e = fast_exp(d);
  return Sums{m, a.z * e, (a.s + fmaxf(d, -1000.0f) * a.z) * e};
}
// The workgroup's sums in every thread: over each wave's lanes, then its waves
// in order; tmp: an entry a wave, free for reuse only after a barrier.
template <int LT>
QL_DEV Sums block_sums(Sums a, Sums *tmp) {
  float m = a.m;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  a = sums_at(a, m);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    a.z += __shfl_xor(a.z, d);
    a.s += __shfl_xor(a.s, d);
  }
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < LT / 64; ++w) m = fmaxf(m, tmp[w].m);
  Sums t{m, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < LT / 64; ++w) {
    const Sums b = sums_at(tmp[w], m);
    t.z += b.z;
    t.s += b.s;
  }
  return t;
}

// A workgroup holds one chunk of a row (the whole row where it fits) in
// registers, R 16-byte pieces a thread, all loaded before the first is used:
// the row is read once from memory. The sums are taken piece by piece as the
// pieces arrive, against the thread's maximum so far (one exponential per
// logit and one per piece to rescale), and the alternatives are found in the
// same registers. Chunks of a split row leave (m, z, s) and their best for
// logprobs_join_kernel.
//
// Alternatives: the top-th largest of 64 disjoint groups' maxima is a lower
// bound of the top-th largest logit (that many groups hold one at least as
// large), so only logits that reach it are listed, typically little more than
// top of them, and ranked among themselves. Keys of value and index are
// distinct, so ties need no further rule. A chunk with NaN or +inf, or one
// whose list would overflow (its largest logits crowded into few threads),
// takes one workgroup maximum per alternative instead.
template <bool F32, int R, bool TOP, int LT>
__global__ __launch_bounds__(LT) void logprobs_kernel(LpArgs g) {
  constexpr int E = lp_elems<F32>();
  constexpr uint32_t FILL = F32 ? 0xff800000u : 0xff80ff80u;   // -inf
  __shared__ Sums ts[LT / 64];
  __shared__ uint64_t tk[LT / 64];
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (uint32_t)g.nchunk;
  const int c = (int)(blockIdx.x % (uint32_t)g.nchunk);
  const void *row = row_of<F32>(g.x, i, g.ld);
  const int64_t j0 = c * g.chunk;
  const int len = (int)min(g.chunk, g.V - j0);
  const int nvec = len / E, rem = len % E;   // rem: the row's end only
  u32x4 x[R];
  float xt = load1<F32>(row, j0 + min(nvec * E + tid, len - 1));
  if (nvec) {
    // pieces past the end re-read the last one (no branch around a load)
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = load16<F32>(row, j0 + E * min(r * LT + tid, nvec - 1));
  }
  Sums a{-FLT_MAX, 0.0f, 0.0f};
  auto add = [&](float v) {
    const float t = v - a.m, e = fast_exp(t);
    a.z += e;
    a.s = fmaf(e, fmaxf(t, -1000.0f), a.s);   // e is 0 below that; keeps 0 * -inf out of s
  };
  float vm = -INFINITY;   // the pieces' maximum itself,
  int best_r = 0;         // and the first piece that holds it
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if ((r + 1) * LT > nvec) {   // uniform
#pragma unroll
      for (int q = 0; q < 4; ++q) x[r][q] = r * LT + tid < nvec ? x[r][q] : FILL;
    }
    if (r * LT < nvec) {
      float pm = fmaxf(elem<F32>(x[r], 0), elem<F32>(x[r], 1));
#pragma unroll
      for (int e = 2; e < E; e += 2)
        pm = fmaxf(pm, fmaxf(elem<F32>(x[r], e), elem<F32>(x[r], e + 1)));
      if (TOP) {
        best_r = pm > vm ? r : best_r;
        vm = fmaxf(vm, pm);
      }
      a = sums_at(a, fmaxf(a.m, pm));
#pragma unroll
      for (int e = 0; e < E; ++e) add(elem<F32>(x[r], e));
    }
  }
  xt = tid < rem ? xt : -INFINITY;
  a = sums_at(a, fmaxf(a.m, xt));
  add(xt);
  const Sums t = block_sums<LT>(a, ts);
  const bool whole = g.nchunk == 1;
  const bool empty = t.z == 0.0f;            // every logit -inf
  const float m = empty ? -INFINITY : t.m, z = t.z;
  const float l = empty ? 0.0f : logf(z);
  if (tid == 0) {
    if (whole)
      finish_row<F32>(g, i, row, m, l, z, t.s, empty);
    else
      g.part[i * g.nchunk + c] = make_float4(t.m, z, t.s, 0.0f);
  }
  if (!TOP) return;

  __shared__ uint64_t list[LP_LIST];
  __shared__ uint64_t grp[LP_GROUPS];
  __shared__ int count;
  const int top = g.top;
  uint64_t *keys = whole ? nullptr : g.keys + (i * g.nchunk + c) * top;
  auto emit = [&](int q, uint64_t key) {
    if (whole)
      put_top(g, i, q, key, m, l, empty);
    else
      keys[q] = key;
  };
  const uint32_t jt = (uint32_t)(j0 + nvec * E + tid);
  uint32_t jb = (uint32_t)(j0 + E * tid);   // index of the thread's first logit
  auto index = [&](int r, int e) { return jb + (uint32_t)(E * LT * r + e); };
  // each pass unpacks the pieces again: kept unpacked, or with every index
  // formed ahead, they would fill the registers
  auto repack = [&]() {
    asm("" : "+v"(jb));
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w = x[r][q];
        asm("" : "+v"(w));
        x[r][q] = w;
      }
  };
  bool plain = z == z;
  repack();
  if (plain) {   // uniform
    // the thread's best: the first place of its maximum in that piece, or the
    // row's end (whose index is the largest)
    u32x4 w = x[0];
#pragma unroll
    for (int r = 1; r < R; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = best_r == r ? x[r][q] : w[q];
    int be = 0;
#pragma unroll
    for (int e = E - 1; e >= 0; --e) be = elem<F32>(w, e) == vm ? e : be;
    uint64_t mine = 0;
    if (tid < nvec) mine = order_key(vm, index(0, 0) + (uint32_t)(E * LT * best_r + be));
    if (tid < rem) mine = OpMax()(mine, order_key(xt, jt));
    uint64_t gm = mine;
#pragma unroll
    for (int d = 1; d < LT / LP_GROUPS; d <<= 1) gm = OpMax()(gm, (uint64_t)__shfl_xor(gm, d));
    if (tid % (LT / LP_GROUPS) == 0) grp[tid / (LT / LP_GROUPS)] = gm;
    if (tid == 0) count = 0;
    __syncthreads();
    // every wave ranks the 64 maxima, one per lane; empty groups are all last
    const uint64_t own = grp[tid & 63];
    int rank = 0;
#pragma unroll 16
    for (int o = 0; o < LP_GROUPS; ++o) rank += grp[o] > own ? 1 : 0;
    const uint64_t hit = __ballot(rank == top - 1 && own != 0);
    const uint64_t floor_key = hit ? __shfl(own, __builtin_ctzll(hit)) : 1;
    const float floor_val = hit ? key_value(floor_key) : -INFINITY;
    repack();
    if (mine >= floor_key) {
      auto offer = [&](float v, uint32_t j) {
        const uint64_t k = order_key(v, j);
        if (k < floor_key) return;
        const int at = atomicAdd(&count, 1);
        if (at < LP_LIST) list[at] = k;
      };
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * LT + tid < nvec) {
          float pm = elem<F32>(x[r], 0);
#pragma unroll
          for (int e = 1; e < E; ++e) pm = fmaxf(pm, elem<F32>(x[r], e));
          if (pm >= floor_val) {   // few pieces
#pragma unroll
            for (int e = 0; e < E; ++e) offer(elem<F32>(x[r], e), index(r, e));
          }
        }
      if (tid < rem) offer(xt, jt);
    }
    __syncthreads();
    plain = count <= LP_LIST;
    if (plain) {
      emit_ranked<LT>(list, count, top, emit);
      for (int q = count + tid; q < top; q += LT) emit(q, 0);   // a chunk of fewer logits
    }
  }
  if (!plain) {
    uint64_t last = ~0ull;
    for (int q = 0; q < top; ++q) {
      uint64_t best = 0;
      repack();
      auto offer = [&](float v, uint32_t j) {
        const uint64_t k = order_key(v, j);
        if (k < last && k > best) best = k;
      };
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * LT + tid < nvec) {
#pragma unroll
          for (int e = 0; e < E; ++e) offer(elem<F32>(x[r], e), index(r, e));
        }
      if (tid < rem) offer(xt, jt);
      last = block_reduce<LT>(best, tk, OpMax());
      if (tid == 0) emit(q, last);
    }
  }
}

// Joins the chunks of a row: sums rescaled to the row's maximum, in a fixed
// order; of the chunks' ordered lists, those keys that reach the smallest
// ceil(top / nchunk)-th entry (at least top keys do) are ranked as above.
template <bool F32>
__global__ __launch_bounds__(JT) void logprobs_join_kernel(LpArgs g) {
  __shared__ Sums ts[JT / 64];
  __shared__ uint64_t tk[JT / 64];
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x;
  const void *row = row_of<F32>(g.x, i, g.ld);
  const float4 *part = g.part + i * g.nchunk;
  Sums a{-FLT_MAX, 0.0f, 0.0f};
  for (int c = tid; c < g.nchunk; c += JT) {
    const float4 p = part[c];
    const float m = fmaxf(a.m, p.x);
    a = sums_at(a, m);
    const Sums b = sums_at(Sums{p.x, p.y, p.z}, m);
    a.z += b.z;
    a.s += b.s;
  }
  const Sums t = block_sums<JT>(a, ts);
  const bool empty = t.z == 0.0f;
  const float m = empty ? -INFINITY : t.m, l = empty ? 0.0f : logf(t.z);
  if (tid == 0) finish_row<F32>(g, i, row, m, l, t.z, t.s, empty);
  const int top = g.top;
  if (!top) return;

  __shared__ uint64_t list[LP_LIST];
  __shared__ int count;
  const int total = g.nchunk * top;                // at most 2^17 chunks of 32
  const uint64_t *keys = g.keys + i * total;
  const int depth = (top + g.nchunk - 1) / g.nchunk;
  uint64_t low = ~0ull;
  for (int c = tid; c < g.nchunk; c += JT) low = min(low, keys[c * top + depth - 1]);
  low = ~block_reduce<JT>(~low, tk, OpMax());
  if (low == 0) low = 1;                           // a short last chunk: every key
  if (tid == 0) count = 0;
  __syncthreads();
  for (int o = tid; o < total; o += JT) {
    const uint64_t k = keys[o];
    if (k < low) continue;
    const int at = atomicAdd(&count, 1);
    if (at < LP_LIST) list[at] = k;
  }
  __syncthreads();
  if (count <= LP_LIST) {
    emit_ranked<JT>(list, count, top,
                [&](int q, uint64_t key) { put_top(g, i, q, key, m, l, empty); });
    return;
  }
  uint64_t last = ~0ull;
  for (int q = 0; q < top; ++q) {
    uint64_t best = 0;
    for (int o = tid; o < total; o += JT) {
      const uint64_t k = keys[o];
      if (k < last && k > best) best = k;
    }
    last = block_reduce<JT>(best, tk, OpMax());
    if (tid == 0) put_top(g, i, q, last, m, l, empty);
  }
}

struct LpGradArgs {
  const void *x;
  int64_t N, V, ld, ldo;
  const int64_t *targets;
  const float *stats, *entropy, *dlp, *dent;
  void *dx;
  int nchunk;
};

template <bool F32, bool NTS>
QL_DEV void store16(void *row, int64_t j, const u32x4 &v) {
  if (F32 && NTS)
    __builtin_nontemporal_store(v, (u32x4_a4 *)((float *)row + j));
  else if (F32)
    *(u32x4_a4 *)((float *)row + j) = v;
  else if (NTS)
    __builtin_nontemporal_store(v, (u32x4_a2 *)((uint16_t *)row + j));
  else
    *(u32x4_a2 *)((uint16_t *)row + j) = v;
}
template <bool F32>
QL_DEV void store1(void *row, int64_t j, float v) {
  if (F32)
    ((float *)row)[j] = v;
  else
    ((uint16_t *)row)[j] = ql::f_to_bf16(v);
}

constexpr int LG_R = 2;   // pieces a thread of the gradient kernel holds

// One read and one write of each logit; the time is that of the bytes. A
// thread loads its pieces before it writes any, and owns what it writes, so
// the gradient may replace the logits. The target's element is written once
// more by the thread that owns it (stores of a thread to one address keep
// their order), which keeps a comparison out of every other element.
template <bool F32, bool ENT, bool NTS>
__global__ __launch_bounds__(JT) void logprobs_grad_kernel(LpGradArgs g) {
  constexpr int E = lp_elems<F32>();
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (uint32_t)g.nchunk;
  const int c = (int)(blockIdx.x % (uint32_t)g.nchunk);
  const void *row = row_of<F32>(g.x, i, g.ld);
  void *out = (void *)row_of<F32>(g.dx, i, g.ldo);
  const int64_t j0 = (int64_t)c * (JT * E * LG_R);
  const int len = (int)min<int64_t>(JT * E * LG_R, g.V - j0);
  const int nvec = len / E, rem = len % E;
  const int64_t t = g.targets[i];
  const float gl = (t >= 0 && t < g.V) ? g.dlp[i] : 0.0f;
  const float ge = ENT ? g.dent[i] : 0.0f;
  const float ent = ENT ? g.entropy[i] : 0.0f;
  const float m = g.stats[2 * i], l = g.stats[2 * i + 1];
  if ((gl == 0.0f && ge == 0.0f) || (m == -INFINITY && l == 0.0f)) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int r = 0; r < LG_R; ++r)
      if (r * JT + tid < nvec) store16<F32, NTS>(out, j0 + E * (r * JT + tid), zero);
    if (tid < rem) store1<F32>(out, j0 + nvec * E + tid, 0.0f);
    return;
  }
  u32x4 x[LG_R];
  if (nvec) {
#pragma unroll
    for (int r = 0; r < LG_R; ++r) x[r] = load16<F32>(row, j0 + E * min(r * JT + tid, nvec - 1));
  }
  const float xt = load1<F32>(row, j0 + min(nvec * E + tid, len - 1));   // used if tid < rem
  const int64_t tl = t - j0;   // the target's place in the chunk, if it has one
  const bool owner = gl != 0.0f && tl >= 0 && tl < len &&
                     tid == (tl < nvec * E ? (int)(tl / E) % JT : (int)tl - nvec * E);
  const float xo = load1<F32>(row, owner ? t : j0);
  auto grad = [&](float v) {   // without the target's own term
    const float lp = (v - m) - l;
    const float p = fast_exp(lp);
    return ENT ? -p * (gl + ge * (fmaxf(lp, -1000.0f) + ent)) : -p * gl;
  };
#pragma unroll
  for (int r = 0; r < LG_R; ++r) {
    const int v = r * JT + tid;
    if (v >= nvec) continue;
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = F32 ? __float_as_uint(grad(elem<F32>(x[r], q)))
                 : ql::pack_bf16x2(grad(elem<F32>(x[r], 2 * q % E)),
                                   grad(elem<F32>(x[r], (2 * q + 1) % E)));
    store16<F32, NTS>(out, j0 + E * v, o);
  }
  if (tid < rem) store1<F32>(out, j0 + nvec * E + tid, grad(xt));
  if (owner) store1<F32>(out, t, grad(xo) + gl);
}

constexpr int64_t kMaxV = (int64_t(1) << 31) - (1 << 16);
constexpr int64_t kMaxThreads = 0xffffffff;   // of one launch

qlora_status check_logits(const qlora_logits *x) {
  if (!x || x->N < 1 || x->V < 1 || x->ld < x->V || !x->data || !aligned16(x->data))
    return QLORA_ERR_INVALID_ARG;
  if (x->dtype != QLORA_DTYPE_BF16 && x->dtype != QLORA_DTYPE_F32) return QLORA_ERR_INVALID_ARG;
  if (x->V >= kMaxV || x->N > 0x7fffffff || x->ld > (int64_t(1) << 40))
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// How rows are cut: threads of a workgroup, pieces of a thread, workgroups of a
// row.
struct Split {
  int LT, R;
  int64_t chunk, nchunk;
};

// A row of 4097 to 8192 pieces stays with one workgroup of 512 threads where
// there are 256 rows or more (no join; 333 x 50257 bf16 16.6 us, in two of 256
// threads 18.8; 1024 threads measured no faster than the join). Any other row
// goes to workgroups of 256 threads, 4096 pieces or less each, in the largest
// chunks that give 512 workgroups in all, two a compute unit, or the smallest (256
// pieces): rows of up to 4096 pieces stay whole from 512 rows on.
Split split_of(int64_t N, int64_t V, bool f32) {
  const int64_t e = f32 ? 4 : 8;
  static const int kR[] = {1, 2, 4, 6, 8, 12, 16};
  Split p;
  p.LT = N >= 256 && V > 256 * e * 16 && V <= 512 * e * 16 ? 512 : 256;
  const int64_t unit = p.LT * e;
  int64_t most = std::min<int64_t>(16, ql_cdiv(V, unit));
  while (p.LT == 256 && most > 1 && N * ql_cdiv(V, most * unit) < 512) most = (most + 1) / 2;
  p.nchunk = ql_cdiv(V, most * unit);
  p.chunk = ql_rup(ql_cdiv(V, p.nchunk), 8);
  p.nchunk = ql_cdiv(V, p.chunk);
  p.R = 16;
  for (int i = 6; i >= 0; --i)
    if (kR[i] * unit >= p.chunk) p.R = kR[i];
  return p;
}

template <bool F32, int R, int LT>
void launch_rows(const LpArgs &g, hipStream_t st) {
  const unsigned grid = (unsigned)(g.N * g.nchunk);
  if (g.top)
    logprobs_kernel<F32, R, true, LT><<<grid, LT, 0, st>>>(g);
  else
    logprobs_kernel<F32, R, false, LT><<<grid, LT, 0, st>>>(g);
}
template <bool F32>
void launch_split(const LpArgs &g, const Split &p, hipStream_t st) {
  // 512 threads hold more than half of what they can
  if (p.LT == 512 && p.R <= 12) launch_rows<F32, 12, 512>(g, st);
  else if (p.LT == 512) launch_rows<F32, 16, 512>(g, st);
  else if (p.R == 1) launch_rows<F32, 1, 256>(g, st);
  else if (p.R == 2) launch_rows<F32, 2, 256>(g, st);
  else if (p.R == 4) launch_rows<F32, 4, 256>(g, st);
  else if (p.R == 6) launch_rows<F32, 6, 256>(g, st);
  else if (p.R == 8) launch_rows<F32, 8, 256>(g, st);
  else if (p.R == 12) launch_rows<F32, 12, 256>(g, st);
  else launch_rows<F32, 16, 256>(g, st);
  if (g.nchunk > 1) logprobs_join_kernel<F32><<<(unsigned)g.N, JT, 0, st>>>(g);
}

template <bool F32, bool ENT>
void launch_grad(const LpGradArgs &g, bool nts, hipStream_t st) {
  const unsigned grid = (unsigned)(g.N * g.nchunk);
  if (nts)
    logprobs_grad_kernel<F32, ENT, true><<<grid, JT, 0, st>>>(g);
  else
    logprobs_grad_kernel<F32, ENT, false><<<grid, JT, 0, st>>>(g);
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool aligned8(const void *p) { return ((uintptr_t)p & 7u) == 0; }

}  // namespace

extern "C" {

size_t qlora_token_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t dtype, int32_t top) {
  if (N < 1 || V < 1 || V >= kMaxV || N > 0x7fffffff || top < 0 || top > QLORA_MAX_TOP ||
      top > V || (dtype != QLORA_DTYPE_BF16 && dtype != QLORA_DTYPE_F32))
    return (size_t)-1;
  const Split p = split_of(N, V, dtype == QLORA_DTYPE_F32);
  if (N * p.nchunk * p.LT > kMaxThreads) return (size_t)-1;
  return p.nchunk == 1 ? 0 : (size_t)(N * p.nchunk) * (16 + 8 * (size_t)top);
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
  if (need == (size_t)-1) return QLORA_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, (int64_t)need)) return QLORA_ERR_WORKSPACE;
  const Split p = split_of(x->N, x->V, x->dtype == QLORA_DTYPE_F32);
  float4 *part = (float4 *)ws;
  const LpArgs g{x->data, x->N, x->V, x->ld, targets, logprob, stats, entropy, top, top_logprobs,
                 top_ids, p.chunk, (int)p.nchunk, part,
                 p.nchunk > 1 ? (uint64_t *)(part + x->N * p.nchunk) : nullptr};
  hipStream_t st = (hipStream_t)stream;
  QlProf prof(QLORA_K_LOGPROBS, st);
  if (x->dtype == QLORA_DTYPE_F32)
    launch_split<true>(g, p, st);
  else
    launch_split<false>(g, p, st);
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
  const bool f32 = x->dtype == QLORA_DTYPE_F32;
  const int64_t nchunk = ql_cdiv(x->V, JT * LG_R * (f32 ? 4 : 8));
  if (x->N * nchunk * JT > kMaxThreads) return QLORA_ERR_UNSUPPORTED;
  const LpGradArgs g{x->data, x->N,    x->V,     x->ld,    dx->ld,   targets,
                     stats,   entropy, dlogprob, dentropy, dx->data, (int)nchunk};
  hipStream_t st = (hipStream_t)stream;
  // logits and gradient that do not fit the 256 MB memory-side cache together:
  // the gradient's stores pass it by, so that they do not push out the logits
  // the forward left there (4096 x 32000 bf16, forward and gradient: 107 us
  // against 141; where both fit, 509 x 50257 float32, 53.4 against 52.9)
  const bool nts = 2 * x->N * x->V * (f32 ? 4 : 2) > ((int64_t)256 << 20);
  QlProf prof(QLORA_K_LOGPROBS_GRAD, st);
  if (f32 && dentropy)
    launch_grad<true, true>(g, nts, st);
  else if (f32)
    launch_grad<true, false>(g, nts, st);
  else if (dentropy)
    launch_grad<false, true>(g, nts, st);
  else
    launch_grad<false, false>(g, nts, st);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

}  // extern "C"
