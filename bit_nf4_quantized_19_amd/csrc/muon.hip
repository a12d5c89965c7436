// Orthogonalised momentum step of the LoRA matrices, gfx950.
//
// Per matrix (R = the smaller side, at most 128):
//   m' = beta m + (1 - beta) g,  u = (1 - beta) g + beta m'  or  m',
//   X0 = u / (|u|_F + eps),  X_{j+1} = P_j X_j,  P_j = a I + b S_j + c S_j^2,
//   S_j = X_j X_j^T,  p' = p - lr (scale X_steps + wd p).
// All P_j are polynomials of S_0 and commute with it, so with Q_0 = I
//   Q_{j+1} = P_j Q_j,   S_{j+1} = P_j S_j P_j,   X_steps = Q_steps X0:
// the iteration runs on R x R matrices and u is read twice in all, once for
// S_0 and once for the update, whatever the number of steps. A direction with
// a small singular value grows by `a` a step, and the rounding of S_0 by a^2
// (485- and 235000-fold after five steps of the usual coefficients), so products
// and sums are taken in float64 on the matrix cores (16x16x4): products of two
// float32 are exact there and their sums do not overflow. The caller bounds
// a^(2 steps): S is not formed from X again, so roundings that grow to its own
// size could make it negative, and the iteration run to infinity.
//
// HBM-bound: 10 bytes an element in gram and 16 in apply (14 without Nesterov,
// where u is m'), 20 if nothing were read twice; the matrix work in float64, at
// the peak rate of 79 TFLOP/s, is 0.4 of gram's and of apply's time for 64 ranks.
// A workgroup's elements of a 64-column chunk go through LDS, so
// that memory is read and written in 16-byte pieces whatever the orientation;
// the workgroups of a compute unit hide each other's latency (by their registers
// four of gram and three of apply for wide matrices of 64 ranks, eight up to 16;
// holding the next chunk in registers instead, two a compute unit, took 329 us
// against 300).
// 80 matrices of 64 x 8192 with Nesterov: 298 us a pass (gram 104, iterate 46,
// apply 163; 155 without), 2.8 TB/s of the 20 bytes; one of 16 x 4096: 15 us
// (3.4, 7.2, 3.0); one of 128 x 4096: 141 us, 107 of them the ten launches of its
// steps.
// Three launches: gram (updates the momentum; partial Gram sums of a range of
// the long side), iterate (one workgroup per matrix: joins the partial sums in
// a fixed order, then the steps; more than 64 ranks take two launches a step
// there), apply (Q times u, and the parameters).
#include <type_traits>

#include "kernels.h"

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

QL_DEV f64x4 mfma_f64(double a, double b, const f64x4 &c) {
  // lane l supplies A[l % 16][l / 16] and B[l / 16][l % 16] and holds
  // D[4 i + l / 16][l % 16]: component i is the B operand of rows 4 i .. +3
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

struct MuonArgs {
  float *p, *m;
  const uint16_t *g;
  uint16_t *out;
  int64_t rows, cols, len;   // len: the longer side
  int R, tall;               // tall: element (i, c) of the short and long side at c R + i
  uint32_t magic;            // ceil(2^20 / R): x / R for x < 64 * 128
  int split;                 // workgroups per matrix
  int64_t chunks;            // of CK along the long side
  double *part;              // [n][split][tiles][256]
  double *Q;                 // [n][RP][RP], Q / (|u| + eps)
  double *S, *P, *inv;       // more than 64 ranks: [n][RP][RP], the same (P^T), [n]
  MuonScalars s;
};

constexpr int CK = 64;        // long-side elements of a chunk

// Barrier between the accesses to LDS of a workgroup's waves; loads and stores
// of global memory, which no other thread of the launch reads, stay in flight
// across it.
QL_DEV void lds_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int NB> constexpr int tiles() { return NB * (NB + 1) / 2; }
// Row strides of a chunk in LDS, stored as it lies in memory: wide [i][c], tall
// [c][i]. The matrix cores' operand reads take 16 x 4 elements; the strides put
// them on 64 different banks: gram reads 16 i by 4 c, apply 4 i by 16 c.
template <int NB, bool TALL> constexpr int gram_stride() {
  return !TALL ? CK + 4 : NB == 1 ? 16 : NB <= 5 ? 80 : 144;
}
template <int NB, bool TALL> constexpr int apply_stride() { return TALL ? 16 * NB + 4 : CK + 16; }
template <int NB, bool TALL, int ST> constexpr int chunk_floats() {
  return TALL ? CK * ST : 16 * NB * ST;
}
template <bool TALL, int ST> QL_DEV int place(int i, int c) { return TALL ? c * ST + i : i * ST + c; }

QL_DEV float muon_m(float m, float g, const MuonScalars &s) {
  return __fadd_rn(__fmul_rn(s.beta, m), __fmul_rn(s.c1, g));
}
QL_DEV float muon_u(float m, float g, const MuonScalars &s) {   // m: the updated one
  return s.nesterov ? __fadd_rn(__fmul_rn(s.c1, g), __fmul_rn(s.beta, m)) : m;
}

// A thread's share of a chunk: NB groups of four elements consecutive in
// memory, group 256 j + thread. Groups run along the rows of a wide matrix
// (16 a row) and through the chunk of a tall one. Offsets in a matrix fit 32
// bits (128 x 2^24 elements).
struct Group {
  uint32_t off;   // of the first element in the matrix
  int n;          // elements that exist: 0 .. 4
};
template <int NB, bool TALL>
struct Share {
  uint32_t off[NB];   // of chunk 0
  uint32_t step;      // from chunk to chunk
  QL_DEV explicit Share(const MuonArgs &a) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const uint32_t e = 256 * j + threadIdx.x;
      off[j] = TALL ? 4 * e : (e >> 4) * (uint32_t)a.cols + 4 * (e & 15);
    }
    step = TALL ? CK * (uint32_t)a.R : CK;
  }
  QL_DEV Group group(const MuonArgs &a, int64_t ch, int j) const {
    const int e = 256 * j + (int)threadIdx.x;
    const bool in = TALL ? e < 16 * a.R : (e >> 4) < a.R;
    Group q{off[j] + (uint32_t)ch * step, in ? 4 : 0};
    const int64_t left = a.len - ch * CK;
    if (left < CK) {   // the last chunk
      const int n = TALL ? (int)left * a.R - 4 * e : (int)left - 4 * (e & 15);
      q.n = !in || n < 0 ? 0 : n > 4 ? 4 : n;
    }
    return q;
  }
};
template <bool VEC>
QL_DEV void load4(const float *p, const Group &q, float (&v)[4]) {
  if (VEC) {
    const float4 x = q.n ? *(const float4 *)(p + q.off) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = x < q.n ? p[q.off + x] : 0.0f;
  }
}
template <bool VEC>
QL_DEV void load4(const uint16_t *p, const Group &q, float (&v)[4]) {
  if (VEC) {
    const uint2 x = q.n ? *(const uint2 *)(p + q.off) : make_uint2(0u, 0u);
    v[0] = ql::bf16lo(x.x), v[1] = ql::bf16hi(x.x), v[2] = ql::bf16lo(x.y), v[3] = ql::bf16hi(x.y);
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = x < q.n ? ql::bf16_to_f(p[q.off + x]) : 0.0f;
  }
}
template <bool VEC>
QL_DEV void store4(float *p, const Group &q, const float (&v)[4]) {
  if (VEC) {
    if (q.n) *(float4 *)(p + q.off) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < q.n) p[q.off + x] = v[x];
  }
}
template <bool VEC>
QL_DEV void store4(uint16_t *p, const Group &q, const float (&v)[4]) {
  if (VEC) {
    if (q.n)
      *(uint2 *)(p + q.off) =
          make_uint2(ql::pack_bf16x2(v[0], v[1]), ql::pack_bf16x2(v[2], v[3]));
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < q.n) p[q.off + x] = ql::f_to_bf16(v[x]);
  }
}
// The group's places in the LDS chunk (absent elements of the chunk too: they
// hold zeros), as one 16-byte access where they are consecutive.
template <bool TALL, int ST, class F4, class F1>
QL_DEV void in_lds(const MuonArgs &a, int j, F4 four, F1 one) {
  const int e = 256 * j + threadIdx.x;
  if (e >= 16 * a.R) return;
  if (!TALL) {
    four(place<TALL, ST>(e >> 4, 4 * (e & 15)));
  } else {
    const uint32_t f = 4 * e;
    const int c = (int)(f * a.magic >> 20), i = (int)f - c * a.R;
    if ((a.R & 3) == 0) {
      four(place<TALL, ST>(i, c));
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t fx = f + x;
        const int cx = (int)(fx * a.magic >> 20);
        one(place<TALL, ST>((int)fx - cx * a.R, cx), x);
      }
    }
  }
}
template <bool TALL, int ST>
QL_DEV void put4(const MuonArgs &a, int j, float *s, const float (&v)[4]) {
  in_lds<TALL, ST>(a, j, [&](int at) { *(float4 *)(s + at) = make_float4(v[0], v[1], v[2], v[3]); },
                   [&](int at, int x) { s[at] = v[x]; });
}
template <bool TALL, int ST>
QL_DEV void get4(const MuonArgs &a, int j, const float *s, float (&v)[4]) {
  in_lds<TALL, ST>(a, j, [&](int at) {
    const float4 x = *(const float4 *)(s + at);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  }, [&](int at, int x) { v[x] = s[at]; });
}

// 1 / (|u| + eps) from the trace of u's Gram matrix. Nothing scales a zero u
// (eps = 0: 0 / 0); otherwise |u| is at least 2^-149, so that the square of the
// result stays finite however small eps is.
QL_DEV double inverse_size(double trace, double eps) {
  return trace == 0.0 && eps > 0.0 ? 0.0 : 1.0 / (sqrt(trace) + eps);
}

template <int NB, bool TALL, bool VEC>
__global__ __launch_bounds__(256) void muon_gram_kernel(MuonArgs a) {
  constexpr int ST = gram_stride<NB, TALL>(), LN = chunk_floats<NB, TALL, ST>();
  __shared__ __align__(16) float s_u[LN];
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.y, base = mat * a.rows * a.cols;
  const int64_t lo = blockIdx.x * a.chunks / a.split, hi = (blockIdx.x + 1) * a.chunks / a.split;
  float *const m = a.m + base;
  const uint16_t *const g = a.g + base;
  // few tiles: the waves share the chunk's columns; many: the tiles
  constexpr bool BYK = NB < 4;
  constexpr int NT = tiles<NB>(), MY = BYK ? NT : (NT + 3) / 4;
  f64x4 acc[MY];
#pragma unroll
  for (int t = 0; t < MY; ++t) acc[t] = f64x4{0.0, 0.0, 0.0, 0.0};
  // the padding of the smaller side stays zero
  for (int e = threadIdx.x; e < LN; e += 256) s_u[e] = 0.0f;
  const Share<NB, TALL> mine(a);
  float mv[NB][4], gv[NB][4];
  auto fetch = [&](int64_t ch) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const Group q = mine.group(a, ch, j);
      load4<VEC>(m, q, mv[j]);
      load4<VEC>(g, q, gv[j]);
    }
  };
  // the chunk's products; W: the wave, whose tiles are known at compile time
  auto sums = [&](auto w) {
    constexpr int W = decltype(w)::value;
#pragma unroll
    for (int s = 0; s < (BYK ? 4 : 16); ++s) {
      const int k = 4 * (BYK ? 4 * wave + s : s) + k4;
      double u[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) u[b] = (double)s_u[place<TALL, ST>(16 * b + c16, k)];
      int t = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = i; j < NB; ++j, ++t)
          if (BYK || t % 4 == W) {
            f64x4 &c = acc[BYK ? t : t / 4];
            c = mfma_f64(u[i], u[j], c);
          }
    }
  };
  for (int64_t ch = lo; ch < hi; ++ch) {
    fetch(ch);
    lds_sync();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float u[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mv[j][x] = muon_m(mv[j][x], gv[j][x], a.s);
        u[x] = muon_u(mv[j][x], gv[j][x], a.s);
      }
      put4<TALL, ST>(a, j, s_u, u);
      store4<VEC>(m, mine.group(a, ch, j), mv[j]);
    }
    lds_sync();
    if (BYK || wave == 0) sums(std::integral_constant<int, 0>());
    else if (wave == 1) sums(std::integral_constant<int, 1>());
    else if (wave == 2) sums(std::integral_constant<int, 2>());
    else sums(std::integral_constant<int, 3>());
  }
  double *part = a.part + (mat * a.split + blockIdx.x) * NT * 256;
  if (BYK) {   // the waves' sums, in their order
    double *red = (double *)s_u;
    static_assert(!BYK || NT * 256 * 8 <= LN * 4, "the chunk's LDS holds the tiles");
    for (int w = 0; w < 4; ++w) {
      lds_sync();
      if (wave != w) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = t * 256 + q * 64 + lane;
          const double v = w ? red[at] + acc[t][q] : acc[t][q];
          if (w < 3) red[at] = v;
          else part[at] = v;
        }
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t % 4 == wave)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[t * 256 + q * 64 + lane] = acc[t / 4][q];
  }
}

// Threads of the iterate kernel: a wave per 16 columns, and more to join the
// partial sums (the others wait).
template <int NB> constexpr int iterate_threads() { return NB == 1 ? 1024 : 512; }

template <int NB>
__global__ __launch_bounds__(iterate_threads<NB>()) void muon_iterate_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB, LS = RP + 2, NT = tiles<NB>(), NTH = iterate_threads<NB>();
  __shared__ double s_a[RP * LS];
  __shared__ double s_j[NB == 1 ? 4 * 256 : 1];
  __shared__ double s_tr;
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.x;
  const double *part = a.part + mat * a.split * NT * 256;
  // Partial sums x0 .. x1 - 1 of the thread's E elements e0, e0 + NTH, ..., the
  // loads of XB of them in flight.
  constexpr int E = NB == 1 ? 1 : (NT * 256 + NTH - 1) / NTH, XB = E > 3 ? 8 : 16;
  auto join = [&](int e0, int x0, int x1, double (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0.0;
    for (int x = x0; x < x1; x += XB) {
      double y[E][XB];
#pragma unroll
      for (int i = 0; i < E; ++i)
#pragma unroll
        for (int h = 0; h < XB; ++h) {
          const int e = e0 + i * NTH;
          y[i][h] = x + h < x1 && e < NT * 256 ? part[(int64_t)(x + h) * NT * 256 + e] : 0.0;
        }
#pragma unroll
      for (int h = 0; h < XB; ++h)
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += y[i][h];
    }
  };
  auto place_sum = [&](int e, double v) {
    int t = e >> 8, i = 0;
    while (t >= NB - i) t -= NB - i, ++i;
    const int row = 16 * i + 4 * ((e >> 6) & 3) + ((e & 63) >> 4), col = 16 * (i + t) + (e & 15);
    s_a[row * LS + col] = v;
    if (t) s_a[col * LS + row] = v;
  };
  if (NB == 1) {   // four quarters of the partial sums at once
    const int y = threadIdx.x >> 8;
    double v[E];
    join(threadIdx.x & 255, y * a.split / 4, (y + 1) * a.split / 4, v);
    s_j[threadIdx.x] = v[0];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int e = threadIdx.x;
      place_sum(e, s_j[e] + s_j[256 + e] + s_j[512 + e] + s_j[768 + e]);
    }
  } else {
    double v[E];
    join(threadIdx.x, 0, a.split, v);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((int)threadIdx.x + i * NTH < NT * 256) place_sum(threadIdx.x + i * NTH, v[i]);
  }
  __syncthreads();
  if (wave == 0) {
    double tr = 0.0;
    for (int i = lane; i < RP; i += 64) tr += s_a[i * LS + i];
    for (int o = 32; o; o >>= 1) tr += __shfl_xor(tr, o);
    if (lane == 0) s_tr = tr;
  }
  __syncthreads();
  const double inv = inverse_size(s_tr, a.s.eps);
  for (int e = threadIdx.x; e < RP * LS; e += NTH) s_a[e] *= inv * inv;
  __syncthreads();

  // wave w < NB holds columns 16 w .. +15 of S and Q as B operands
  const bool on = wave < NB;
  double sp[NB * 4], qp[NB * 4];
#pragma unroll
  for (int x = 0; x < NB * 4; ++x) {
    const int row = 4 * x + k4, col = 16 * wave + c16;
    sp[x] = on ? s_a[row * LS + col] : 0.0;
    qp[x] = row == col ? 1.0 : 0.0;
  }
  auto times = [&](const double (&in)[NB * 4], double (&out)[NB * 4]) {   // (LDS matrix) * in
    f64x4 d[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) d[b] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int x = 0; x < NB * 4; ++x) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        d[b] = mfma_f64(s_a[(16 * b + c16) * LS + 4 * x + k4], in[x], d[b]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) out[4 * b + q] = d[b][q];
  };
  if (NB == 1 && !on) return;   // the steps of one block need one wave and no barrier
  auto sync = [&] {
    if (NB > 1) {
      __syncthreads();
    } else {   // LDS accesses of a wave are in order: keep the compiler to it
      asm volatile("" ::: "memory");
      __builtin_amdgcn_wave_barrier();
    }
  };
  auto store = [&](const double (&v)[NB * 4]) {
    sync();
    if (on)
#pragma unroll
      for (int x = 0; x < NB * 4; ++x) s_a[(4 * x + k4) * LS + 16 * wave + c16] = v[x];
    sync();
  };
#pragma clang loop unroll(disable)
  for (int step = 0; step < a.s.steps; ++step) {
    double t[NB * 4];
    if (on) {
      times(sp, t);
#pragma unroll
      for (int x = 0; x < NB * 4; ++x)
        t[x] = (4 * x + k4 == 16 * wave + c16 ? a.s.a : 0.0) + a.s.b * sp[x] + a.s.c * t[x];
    }
    store(t);
    const bool more = step + 1 < a.s.steps;
    if (on) {
      if (step == 0) {
#pragma unroll
        for (int x = 0; x < NB * 4; ++x) qp[x] = t[x];
      } else {
        times(qp, qp);
      }
      if (more) {
        times(sp, t);
        times(t, sp);
      }
    }
    if (more) store(sp);
  }
  double *Q = a.Q + mat * RP * RP;
  if (on)
#pragma unroll
    for (int x = 0; x < NB * 4; ++x) Q[(4 * x + k4) * RP + 16 * wave + c16] = qp[x] * inv;
}

// ---- more than 64 ranks: a workgroup per 16 columns ------------------------------
// One compute unit takes 232 us for the 17 products of 128 x 128 in float64, so
// the columns of a matrix are dealt to NB workgroups and a step is two
// launches: poly (P from all of S) and advance (the workgroup's columns of Q
// and S from all of P). Both read their left operand from L2 by rows, that is
// transposed: S as it is, symmetric up to rounding, P from where poly put its
// transpose. The difference matters there: with P^T for P, Q comes out as the
// transpose of what apply, which reads its columns as rows, can use. Rounding
// then grew by a^3 a step (the update of a rank-one 80 x 300 off by 9e-5 after
// eight steps and 0.15 after ten, of a size of one; so 3e-8, the rounding of the
// float32 parameters, after either).
// Partial sums of one 16 x 16 tile and its mirror image, in order.
template <int NB>
__global__ __launch_bounds__(256) void muon_join_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB, NT = tiles<NB>();
  const int e = threadIdx.x;
  const int64_t mat = blockIdx.y;
  const double *part = a.part + (mat * a.split * NT + blockIdx.x) * 256 + e;
  double v = 0.0;
#pragma unroll 8
  for (int x = 0; x < a.split; ++x) v += part[(int64_t)x * NT * 256];
  int t = (int)blockIdx.x, i = 0;
  while (t >= NB - i) t -= NB - i, ++i;
  const int row = 16 * i + 4 * (e >> 6) + ((e & 63) >> 4), col = 16 * (i + t) + (e & 15);
  double *S = a.S + mat * RP * RP;
  S[row * RP + col] = v;
  if (t) S[col * RP + row] = v;
}

// inverse_size of the matrix whose Gram sums are S.
template <int NB>
QL_DEV double inverse_size(const MuonArgs &a, const double *S) {
  constexpr int RP = 16 * NB;
  double tr = 0.0;   // every wave for itself, in the same order
  for (int i = threadIdx.x & 63; i < RP; i += 64) tr += S[i * RP + i];
  for (int o = 32; o; o >>= 1) tr += __shfl_xor(tr, o);
  return inverse_size(tr, a.s.eps);
}
// Row blocks wave and wave + 4 of (rows of L) times the panel in LDS.
template <int NB>
QL_DEV void panel_product(const double *L, const double *panel, f64x4 (&d)[2]) {
  constexpr int RP = 16 * NB;
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b1 = wave + 4 < NB ? wave + 4 : wave;   // past the end: computed, not used
  d[0] = d[1] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
  for (int x = 0; x < NB * 4; ++x) {
    const double *l = L + (4 * x + k4) * RP + c16, y = panel[(4 * x + k4) * 16 + c16];
    d[0] = mfma_f64(l[16 * wave], y, d[0]);
    d[1] = mfma_f64(l[16 * b1], y, d[1]);
  }
}

template <int NB>
__global__ __launch_bounds__(256) void muon_poly_kernel(MuonArgs a, int first) {
  constexpr int RP = 16 * NB;
  __shared__ double s_b[RP * 16];
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t mat = blockIdx.y;
  const int col = 16 * (int)blockIdx.x;
  const double *S = a.S + mat * RP * RP;
  double sc = 1.0;
  if (first) {   // S holds the Gram sums: S_0 is inv^2 times them
    const double inv = inverse_size<NB>(a, S);
    sc = inv * inv;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.inv[mat] = inv;
  }
  for (int e = threadIdx.x; e < RP * 16; e += 256)
    s_b[e] = sc * S[(e >> 4) * RP + col + (e & 15)];
  __syncthreads();
  f64x4 d[2];
  panel_product<NB>(S, s_b, d);
  double *P = a.P + mat * RP * RP;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int b = wave + 4 * r;
    if (b >= NB) break;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int row = 16 * b + 4 * q + k4;
      P[(col + c16) * RP + row] = (row == col + c16 ? a.s.a : 0.0) +   // transposed
                                  a.s.b * s_b[row * 16 + c16] + a.s.c * (sc * d[r][q]);
    }
  }
}

template <int NB>
__global__ __launch_bounds__(256) void muon_advance_kernel(MuonArgs a, int first, int last) {
  constexpr int RP = 16 * NB;
  __shared__ double s_b[RP * 16];
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t mat = blockIdx.y;
  const int col = 16 * (int)blockIdx.x;
  const double *P = a.P + mat * RP * RP;
  double *S = a.S + mat * RP * RP, *Q = a.Q + mat * RP * RP;
  const double inv = a.inv[mat];
  f64x4 d[2];
  // Q' = P Q (the first Q is the identity), times 1 / (|u| + eps) at the end
  if (!first) {
    for (int e = threadIdx.x; e < RP * 16; e += 256) s_b[e] = Q[(e >> 4) * RP + col + (e & 15)];
    __syncthreads();
    panel_product<NB>(P, s_b, d);
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int b = wave + 4 * r;
    if (b >= NB) break;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = (16 * b + 4 * q + k4) * RP + col + c16;
      const double v = first ? P[at] : d[r][q];   // the first P: symmetric to a rounding
      Q[at] = last ? v * inv : v;
    }
  }
  if (last) return;
  // S' = P (P S)
  const double sc = first ? inv * inv : 1.0;
  for (int e = threadIdx.x; e < RP * 16; e += 256)
    s_b[e] = sc * S[(e >> 4) * RP + col + (e & 15)];
  __syncthreads();
  panel_product<NB>(P, s_b, d);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (wave + 4 * r < NB)
#pragma unroll
      for (int q = 0; q < 4; ++q) s_b[(16 * (wave + 4 * r) + 4 * q + k4) * 16 + c16] = d[r][q];
  __syncthreads();
  panel_product<NB>(P, s_b, d);
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (wave + 4 * r < NB)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        S[(16 * (wave + 4 * r) + 4 * q + k4) * RP + col + c16] = d[r][q];
}

// No steps: Q is the identity over |u| + eps.
template <int NB>
__global__ __launch_bounds__(256) void muon_no_steps_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB;
  const int64_t mat = blockIdx.x;
  const double inv = inverse_size<NB>(a, a.S + mat * RP * RP);
  for (int e = threadIdx.x; e < RP * RP; e += 256)
    a.Q[mat * RP * RP + e] = e / RP == e % RP ? inv : 0.0;
}

template <int NB, bool TALL, bool VEC>
__global__ __launch_bounds__(256) void muon_apply_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB, ST = apply_stride<NB, TALL>(), LN = chunk_floats<NB, TALL, ST>();
  __shared__ __align__(16) float s_u[LN];
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.y, base = mat * a.rows * a.cols;
  const int64_t lo = blockIdx.x * a.chunks / a.split, hi = (blockIdx.x + 1) * a.chunks / a.split;
  float *const p = a.p + base;
  const float *const m = a.m + base;
  const uint16_t *const g = a.g + base;
  uint16_t *const out = a.out + base;
  // The wave's rows of Q stay in registers. Up to three row blocks: all of
  // them, times 16 of the chunk's columns; more: every fourth row block, times
  // all columns.
  constexpr bool BYC = NB < 4;
  constexpr int RB = BYC ? NB : (NB + 3) / 4, CB = BYC ? 1 : CK / 16;
  double q[RB][NB * 4];
  {
    const double *Q = a.Q + mat * RP * RP;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int b = BYC ? r : wave + 4 * r < NB ? wave + 4 * r : wave;   // Q is symmetric up to
#pragma unroll
      for (int x = 0; x < NB * 4; ++x) q[r][x] = Q[(4 * x + k4) * RP + 16 * b + c16];   // rounding
    }
  }
  for (int e = threadIdx.x; e < LN; e += 256) s_u[e] = 0.0f;
  const Share<NB, TALL> mine(a);
  float mv[NB][4], gv[NB][4], pv[NB][4];
  auto fetch = [&](int64_t ch) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      Group x = mine.group(a, ch, j);
      load4<VEC>(m, x, mv[j]);
      // without Nesterov u is m'; a mask, as a branch around the loads parted
      // them from m's and took 172 us, not 157
      x.n = a.s.nesterov ? x.n : 0;
      load4<VEC>(g, x, gv[j]);
    }
  };
  for (int64_t ch = lo; ch < hi; ++ch) {
    fetch(ch);
    lds_sync();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float u[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) u[x] = muon_u(mv[j][x], gv[j][x], a.s);
      put4<TALL, ST>(a, j, s_u, u);
      load4<VEC>((const float *)p, mine.group(a, ch, j), pv[j]);
    }
    lds_sync();
    f64x4 d[CB][RB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int r = 0; r < RB; ++r) d[c][r] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int x = 0; x < NB * 4; ++x)
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const double u = (double)s_u[place<TALL, ST>(4 * x + k4, 16 * (BYC ? wave : c) + c16)];
#pragma unroll
        for (int r = 0; r < RB; ++r) d[c][r] = mfma_f64(q[r][x], u, d[c][r]);
      }
    lds_sync();
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int b = BYC ? r : wave + 4 * r;
        if (b >= NB) continue;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s_u[place<TALL, ST>(16 * b + 4 * x + k4, 16 * (BYC ? wave : c) + c16)] = (float)d[c][r][x];
      }
    lds_sync();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const Group x = mine.group(a, ch, j);
      float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      get4<TALL, ST>(a, j, s_u, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float dir = __fadd_rn(__fmul_rn(a.s.scale, o[i]), __fmul_rn(a.s.wd, pv[j][i]));
        o[i] = __fsub_rn(pv[j][i], __fmul_rn(a.s.lr, dir));
      }
      store4<VEC>(p, x, o);
      store4<VEC>(out, x, o);
    }
  }
}

struct MuonPlan {
  int R, NB, split;
  int64_t len, chunks, part, q, inv;   // part, q, inv: bytes
};
MuonPlan muon_plan(int64_t n, int64_t rows, int64_t cols) {
  MuonPlan p;
  p.R = (int)(rows < cols ? rows : cols);
  p.len = rows < cols ? cols : rows;
  p.NB = (int)ql_cdiv(p.R, 16);
  p.chunks = ql_cdiv(p.len, CK);
  // four workgroups for each compute unit, also where fewer fit (apply of 64
  // ranks: 960 of 80 matrices on 768 places)
  int64_t s = n < 1024 ? 1024 / n : 1;
  s = s < p.chunks ? s : p.chunks;
  p.split = (int)s;
  p.part = ql_rup(n * s * (p.NB * (p.NB + 1) / 2) * 2048, 256);
  p.q = ql_rup(n * p.NB * p.NB * 2048, 256);
  p.inv = ql_rup(n * 8, 256);
  return p;
}

template <int NB, bool TALL, bool VEC>
void launch_form(const MuonArgs &a, unsigned n, hipStream_t st) {
  const dim3 grid((unsigned)a.split, n);
  muon_gram_kernel<NB, TALL, VEC><<<grid, 256, 0, st>>>(a);
  if constexpr (NB <= 4) {
    muon_iterate_kernel<NB><<<n, iterate_threads<NB>(), 0, st>>>(a);
  } else {
    const dim3 panels(NB, n);
    muon_join_kernel<NB><<<dim3(tiles<NB>(), n), 256, 0, st>>>(a);
    if (a.s.steps == 0) muon_no_steps_kernel<NB><<<n, 256, 0, st>>>(a);
    for (int i = 0; i < a.s.steps; ++i) {
      muon_poly_kernel<NB><<<panels, 256, 0, st>>>(a, i == 0);
      muon_advance_kernel<NB><<<panels, 256, 0, st>>>(a, i == 0, i + 1 == a.s.steps);
    }
  }
  muon_apply_kernel<NB, TALL, VEC><<<grid, 256, 0, st>>>(a);
}
template <int NB>
void launch_nb(const MuonArgs &a, unsigned n, hipStream_t st) {
  // VEC: every group of four elements is aligned, and whole or absent
  const bool vec = (a.tall ? a.rows * a.cols : a.cols) % 4 == 0;
  if (a.tall) {
    if (vec) launch_form<NB, true, true>(a, n, st);
    else launch_form<NB, true, false>(a, n, st);
  } else {
    if (vec) launch_form<NB, false, true>(a, n, st);
    else launch_form<NB, false, false>(a, n, st);
  }
}

}  // namespace

// The workgroups of n matrices are at most max(n, 1024), n times the chunks of one
// at the most; counting that many, the size serves fewer matrices too, which
// may be split further (512 in two each, 600 not at all).
size_t muon_ws_bytes(int64_t n, int64_t rows, int64_t cols) {
  const MuonPlan p = muon_plan(n, rows, cols);
  const int64_t most = n >= 1024 ? n : n * p.chunks < 1024 ? n * p.chunks : 1024;
  const int64_t part = ql_rup(most * (p.NB * (p.NB + 1) / 2) * 2048, 256);
  return (size_t)(part + (p.NB <= 4 ? p.q : 3 * p.q + p.inv));
}

qlora_status launch_muon(float *p, float *m, const uint16_t *g, uint16_t *out, int64_t n,
                         int64_t rows, int64_t cols, const MuonScalars &s, void *ws,
                         hipStream_t st) {
  const MuonPlan pl = muon_plan(n, rows, cols);
  const MuonArgs a{p, m, g, out, rows, cols, pl.len, pl.R, rows > cols,
                   (uint32_t)((1u << 20) + pl.R - 1) / (uint32_t)pl.R, pl.split, pl.chunks,
                   (double *)ws, (double *)((char *)ws + pl.part),
                   (double *)((char *)ws + pl.part + pl.q),
                   (double *)((char *)ws + pl.part + 2 * pl.q),
                   (double *)((char *)ws + pl.part + 3 * pl.q), s};
  QlProf prof(QLORA_K_MUON, st);
  switch (pl.NB) {
    case 1: launch_nb<1>(a, (unsigned)n, st); break;
    case 2: launch_nb<2>(a, (unsigned)n, st); break;
    case 3: launch_nb<3>(a, (unsigned)n, st); break;
    case 4: launch_nb<4>(a, (unsigned)n, st); break;
    case 5: launch_nb<5>(a, (unsigned)n, st); break;
    case 6: launch_nb<6>(a, (unsigned)n, st); break;
    case 7: launch_nb<7>(a, (unsigned)n, st); break;
    default: launch_nb<8>(a, (unsigned)n, st); break;
  }
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}
