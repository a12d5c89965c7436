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
// a small singular value grows by `a` a step, and the rounding of S_0 and Q
// with it (485-fold after five steps of the usual coefficients), so products
// and sums are taken in float64 on the matrix cores (16x16x4): products of two
// float32 are exact there, and nothing overflows.
//
// Three launches: gram (updates the momentum; partial Gram sums of a range of
// the long side), iterate (one workgroup per matrix: joins the partial sums in
// a fixed order, then the steps), apply (Q times u, and the parameters).
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
  MuonScalars s;
};

constexpr int CK = 64;        // long-side elements of a chunk
constexpr int US = CK + 4;    // row stride of a chunk in LDS (64 banks: 4 i + k distinct)

template <int NB> constexpr int tiles() { return NB * (NB + 1) / 2; }

QL_DEV float muon_m(float m, float g, const MuonScalars &s) {
  return __fadd_rn(__fmul_rn(s.beta, m), __fmul_rn(s.c1, g));
}
QL_DEV float muon_u(float m, float g, const MuonScalars &s) {   // m: the updated one
  return s.nesterov ? __fadd_rn(__fmul_rn(s.c1, g), __fmul_rn(s.beta, m)) : m;
}

// Calls f(offset in the matrix, place in the LDS chunk) for every element of
// chunk c0 that exists, each by one thread.
template <class F>
QL_DEV void for_chunk(const MuonArgs &a, int64_t c0, F f) {
  const int w = (int)(a.len - c0 < CK ? a.len - c0 : CK);
  if (!a.tall) {
    for (int e = threadIdx.x; e < a.R * CK; e += blockDim.x) {
      const int i = e / CK, c = e % CK;
      if (c < w) f(i * a.cols + c0 + c, i * US + c);
    }
  } else {
    for (int e = threadIdx.x; e < a.R * w; e += blockDim.x) {
      const int c = (int)((uint32_t)e * a.magic >> 20), i = e - c * a.R;
      f(c0 * a.R + e, i * US + c);
    }
  }
}

template <int NB>
__global__ __launch_bounds__(256) void muon_gram_kernel(MuonArgs a) {
  __shared__ float s_u[16 * NB * US];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.y, base = mat * a.rows * a.cols;
  const int64_t lo = blockIdx.x * a.chunks / a.split, hi = (blockIdx.x + 1) * a.chunks / a.split;
  // few tiles: the waves share the chunk's columns; many: the tiles
  constexpr bool BYK = NB < 4;
  constexpr int NT = tiles<NB>(), MY = BYK ? NT : (NT + 3) / 4;
  f64x4 acc[MY];
#pragma unroll
  for (int t = 0; t < MY; ++t) acc[t] = f64x4{0.0, 0.0, 0.0, 0.0};
  for (int64_t ch = lo; ch < hi; ++ch) {
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * NB * US; e += 256) s_u[e] = 0.0f;
    __syncthreads();
    for_chunk(a, ch * CK, [&](int64_t off, int at) {
      const float g = ql::bf16_to_f(a.g[base + off]);
      const float m = muon_m(a.m[base + off], g, a.s);
      a.m[base + off] = m;
      s_u[at] = muon_u(m, g, a.s);
    });
    __syncthreads();
#pragma unroll
    for (int s = 0; s < (BYK ? 4 : 16); ++s) {
      const int k = 4 * (BYK ? 4 * wave + s : s) + (lane >> 4);
      double u[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) u[b] = (double)s_u[(16 * b + (lane & 15)) * US + k];
      int t = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = i; j < NB; ++j, ++t) {
          if (BYK) acc[t] = mfma_f64(u[i], u[j], acc[t]);
          else if (t % 4 == wave) acc[t / 4] = mfma_f64(u[i], u[j], acc[t / 4]);
        }
    }
  }
  double *part = a.part + ((mat * a.split + blockIdx.x) * (BYK ? 4 : 1)) * NT * 256;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (!BYK && t % 4 != wave) continue;
    double *to = part + ((BYK ? wave * NT : 0) + t) * 256;
#pragma unroll
    for (int q = 0; q < 4; ++q) to[q * 64 + lane] = acc[BYK ? t : t / 4][q];
  }
}

template <int NB>
__global__ __launch_bounds__(64 * NB) void muon_iterate_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB, LS = RP + 2, NT = tiles<NB>();
  __shared__ double s_a[RP * LS];
  __shared__ double s_tr;
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.x;
  const int np = a.split * (NB < 4 ? 4 : 1);
  const double *part = a.part + mat * np * NT * 256;
  for (int e = threadIdx.x; e < NT * 256; e += 64 * NB) {
    double v = 0.0;
    for (int x = 0; x < np; ++x) v += part[(int64_t)x * NT * 256 + e];
    int t = e >> 8, i = 0;
    while (t >= NB - i) t -= NB - i, ++i;
    const int row = 16 * i + 4 * ((e >> 6) & 3) + ((e & 63) >> 4), col = 16 * (i + t) + (e & 15);
    s_a[row * LS + col] = v;
    if (t) s_a[col * LS + row] = v;
  }
  __syncthreads();
  if (wave == 0) {
    double tr = 0.0;
    for (int i = lane; i < RP; i += 64) tr += s_a[i * LS + i];
    for (int o = 32; o; o >>= 1) tr += __shfl_xor(tr, o);
    if (lane == 0) s_tr = tr;
  }
  __syncthreads();
  const double inv = 1.0 / (sqrt(s_tr) + a.s.eps);
  for (int e = threadIdx.x; e < RP * LS; e += 64 * NB) s_a[e] *= inv * inv;
  __syncthreads();

  // wave w holds columns 16 w .. +15 of S and Q as B operands
  double sp[NB * 4], qp[NB * 4];
#pragma unroll
  for (int x = 0; x < NB * 4; ++x) {
    const int row = 4 * x + k4, col = 16 * wave + c16;
    sp[x] = s_a[row * LS + col];
    qp[x] = row == col ? 1.0 : 0.0;
  }
  auto times = [&](const double (&in)[NB * 4], double (&out)[NB * 4]) {   // (LDS matrix) * in
    f64x4 d[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) d[b] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int x = 0; x < NB * 4; ++x)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        d[b] = mfma_f64(s_a[(16 * b + c16) * LS + 4 * x + k4], in[x], d[b]);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) out[4 * b + q] = d[b][q];
  };
  auto store = [&](const double (&v)[NB * 4]) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NB * 4; ++x) s_a[(4 * x + k4) * LS + 16 * wave + c16] = v[x];
    __syncthreads();
  };
#pragma clang loop unroll(disable)
  for (int step = 0; step < a.s.steps; ++step) {
    double t[NB * 4];
    times(sp, t);
#pragma unroll
    for (int x = 0; x < NB * 4; ++x)
      t[x] = (4 * x + k4 == 16 * wave + c16 ? a.s.a : 0.0) + a.s.b * sp[x] + a.s.c * t[x];
    store(t);
    times(qp, qp);
    if (step + 1 < a.s.steps) {
      times(sp, t);
      times(t, sp);
      store(sp);
    }
  }
  double *Q = a.Q + mat * RP * RP;
#pragma unroll
  for (int x = 0; x < NB * 4; ++x) Q[(4 * x + k4) * RP + 16 * wave + c16] = qp[x] * inv;
}

template <int NB>
__global__ __launch_bounds__(256) void muon_apply_kernel(MuonArgs a) {
  constexpr int RP = 16 * NB;
  __shared__ float s_u[RP * US];
  const int lane = threadIdx.x & 63, c16 = lane & 15, k4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mat = blockIdx.y, base = mat * a.rows * a.cols;
  const double *Q = a.Q + mat * RP * RP;
  const int64_t lo = blockIdx.x * a.chunks / a.split, hi = (blockIdx.x + 1) * a.chunks / a.split;
  for (int64_t ch = lo; ch < hi; ++ch) {
    __syncthreads();
    for (int e = threadIdx.x; e < RP * US; e += 256) s_u[e] = 0.0f;
    __syncthreads();
    for_chunk(a, ch * CK, [&](int64_t off, int at) {
      s_u[at] = muon_u(a.m[base + off], ql::bf16_to_f(a.g[base + off]), a.s);
    });
    __syncthreads();
    // wave w: columns 16 w .. +15 of the chunk, all rows
    f64x4 d[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) d[b] = f64x4{0.0, 0.0, 0.0, 0.0};
    for (int x = 0; x < NB * 4; ++x) {
      const double u = (double)s_u[(4 * x + k4) * US + 16 * wave + c16];
#pragma unroll
      for (int b = 0; b < NB; ++b)   // Q is symmetric up to rounding: read by columns
        d[b] = mfma_f64(Q[(int64_t)(4 * x + k4) * RP + 16 * b + c16], u, d[b]);
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s_u[(16 * b + 4 * q + k4) * US + 16 * wave + c16] = (float)d[b][q];
    __syncthreads();
    for_chunk(a, ch * CK, [&](int64_t off, int at) {
      const float p = a.p[base + off];
      const float dir = __fadd_rn(__fmul_rn(a.s.scale, s_u[at]), __fmul_rn(a.s.wd, p));
      const float q = __fsub_rn(p, __fmul_rn(a.s.lr, dir));
      a.p[base + off] = q;
      a.out[base + off] = ql::f_to_bf16(q);
    });
  }
}

struct MuonPlan {
  int R, NB, split;
  int64_t len, chunks, part, q;   // part, q: bytes
};
MuonPlan muon_plan(int64_t n, int64_t rows, int64_t cols) {
  MuonPlan p;
  p.R = (int)(rows < cols ? rows : cols);
  p.len = rows < cols ? cols : rows;
  p.NB = (int)ql_cdiv(p.R, 16);
  p.chunks = ql_cdiv(p.len, CK);
  int64_t s = ql_cdiv(1024, n);
  s = s < p.chunks ? s : p.chunks;
  p.split = (int)s;
  const int64_t np = s * (p.NB < 4 ? 4 : 1);
  p.part = ql_rup(n * np * (p.NB * (p.NB + 1) / 2) * 2048, 256);
  p.q = ql_rup(n * p.NB * p.NB * 2048, 256);
  return p;
}

template <int NB>
void launch_nb(const MuonArgs &a, unsigned n, hipStream_t st) {
  const dim3 grid((unsigned)a.split, n);
  muon_gram_kernel<NB><<<grid, 256, 0, st>>>(a);
  muon_iterate_kernel<NB><<<n, 64 * NB, 0, st>>>(a);
  muon_apply_kernel<NB><<<grid, 256, 0, st>>>(a);
}

}  // namespace

size_t muon_ws_bytes(int64_t n, int64_t rows, int64_t cols) {
  const MuonPlan p = muon_plan(n, rows, cols);
  return (size_t)(p.part + p.q);
}

qlora_status launch_muon(float *p, float *m, const uint16_t *g, uint16_t *out, int64_t n,
                         int64_t rows, int64_t cols, const MuonScalars &s, void *ws,
                         hipStream_t st) {
  const MuonPlan pl = muon_plan(n, rows, cols);
  const MuonArgs a{p, m, g, out, rows, cols, pl.len, pl.R, rows > cols,
                   (uint32_t)((1u << 20) + pl.R - 1) / (uint32_t)pl.R, pl.split, pl.chunks,
                   (double *)ws, (double *)((char *)ws + pl.part), s};
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
