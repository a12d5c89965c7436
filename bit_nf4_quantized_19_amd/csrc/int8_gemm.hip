// Integer GEMM and decode product of the 8-bit base with the LoRA rank-r
// term, gfx950 MFMA.
//
//   forward: Y[m][n]  = sx[m] sw[n] sum_K Wq[n][K] Xq[m][K] + sum_t B[n][t] (sH)[m][t]
//   dX:      dX[m][n] = se[m] sum_K Wq[K][n] Eq[m][K]       + sum_t A[t][n] (sG)[m][t]
//
// The integer sums are exact in int32 (K <= 131072), so how they are split
// does not change a bit of the result. As in the NF4 GEMM the product is
// computed transposed (weights are the MFMA's A operand), so each lane ends
// with 4 consecutive n of one token, and s H (s G) comes as bf16 hi + lo parts.
#include "kernels.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct I8Args {
  const int8_t *W;       // d x k codes
  const float *sw;       // [d]
  int64_t d, k;
  const int8_t *In;      // M x ldi codes, zero past Ktot
  int64_t ldi;           // a multiple of 128
  const float *sx;       // [M]
  int64_t M, Ntot, Ktot;
  const uint16_t *L;     // rank-r term: B (d x r) or A (r x k)
  const uint16_t *Shi, *Slo;   // M x rp
  int r, rp;
  uint16_t *Out;         // M x Ntot
};

QL_DEV uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// LDS DMA: lane l's 16 bytes at gptr land at LDS address lds + 16 l (lds
// wave-uniform, carried by M0, which nothing else here uses).
QL_DEV void dma16(const void *gptr, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(gptr), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
QL_DEV void wait_vm_le() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Workgroup barrier that no memory access moves across; the wave's own LDS
// reads have arrived before it.
QL_DEV void block_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

QL_DEV i32x16 mfma_i8(const i32x4 &a, const i32x4 &b, const i32x16 &c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

constexpr int BK = 128;   // K-step: 128 codes, rows of 128 bytes in LDS

// Chunk (16 bytes) c of K-contiguous tile row `row`: its place in the row,
// permuted so that neighbouring rows' equal chunks lie in different banks.
QL_DEV int swz(int row, int c) { return c ^ ((row ^ (row >> 2)) & 7); }

// MODE 0 forward, 1 dX. BN x BM tile by WN x WM waves, NST LDS stages.
template <int MODE, int BN, int BM, int WN, int WM, int NST>
__global__ __launch_bounds__(64 * WN * WM) void int8_gemm_kernel(I8Args g) {
  constexpr int NW = WN * WM, TI = BN / WN / 32, TJ = BM / WM / 32;
  constexpr int WDMA = BN * BK / 1024 / NW, XDMA = BM * BK / 1024 / NW;
  __shared__ __align__(1024) uint4 s_t[NST * (BN + BM) * BK / 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN, r32 = lane & 31, h = lane >> 5;

  // XCD-aware order of the tiles: workgroups of one XCD (id % 8) take a
  // contiguous range, in groups of 4 token blocks with the column tile slow
  const int64_t tn = ql_cdiv(g.Ntot, BN), tm = ql_cdiv(g.M, BM), nt = tn * tm;
  int64_t id = blockIdx.x;
  {
    const int64_t q = nt / 8, rest = nt % 8, x = id % 8, y = id / 8;
    id = x * q + (x < rest ? x : rest) + y;
  }
  const int64_t g0 = id / (4 * tn) * 4, gm = tm - g0 < 4 ? tm - g0 : 4, in = id - g0 * tn;
  const int64_t n0 = in / gm * BN, m0 = (g0 + in % gm) * BM;

  // this lane's DMA sources (rows and columns past the matrix fetch the last
  // valid ones: their sums are not stored, or meet the zeros of In past Ktot)
  int64_t xoff[XDMA], woff[WDMA];
  int wrow[WDMA];
#pragma unroll
  for (int i = 0; i < XDMA; ++i) {
    const int row = 8 * (XDMA * wave + i) + (lane >> 3);
    const int64_t m = m0 + row < g.M ? m0 + row : g.M - 1;
    xoff[i] = m * g.ldi + 16 * swz(row, lane & 7);
  }
#pragma unroll
  for (int i = 0; i < WDMA; ++i) {
    if (MODE == 0) {
      const int row = 8 * (WDMA * wave + i) + (lane >> 3);
      const int64_t n = n0 + row < g.d ? n0 + row : g.d - 1;
      wrow[i] = 16 * swz(row, lane & 7);
      woff[i] = n * g.k;
    } else {
      constexpr int CPR = BN / 16;   // chunks of a tile row
      const int p = 64 * (WDMA * wave + i) + lane;
      wrow[i] = p / CPR;
      const int c = (p % CPR) ^ (wrow[i] & 7);
      const int64_t n = n0 + 16 * c;
      woff[i] = n < g.k ? n : g.k - 16;
    }
  }
  const int nk = (int)ql_cdiv(g.Ktot, BK);
  auto issue = [&](int step) {
    const int64_t kk = (int64_t)step * BK;
    const uint32_t base = lds_addr(s_t) + (uint32_t)(step % NST) * (BN + BM) * BK;
#pragma unroll
    for (int i = 0; i < WDMA; ++i) {
      const int8_t *src;
      if (MODE == 0) {
        const int64_t c = kk + wrow[i];
        src = g.W + woff[i] + (c < g.k ? c : g.k - 16);
      } else {
        const int64_t j = kk + wrow[i];
        src = g.W + (j < g.d ? j : g.d - 1) * g.k + woff[i];
      }
      dma16(src, base + 1024 * (WDMA * wave + i));
    }
#pragma unroll
    for (int i = 0; i < XDMA; ++i)
      dma16(g.In + xoff[i] + kk, base + BN * BK + 1024 * (XDMA * wave + i));
  };

  i32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

  for (int s = 0; s < NST - 1 && s < nk; ++s) issue(s);
  for (int step = 0; step < nk; ++step) {
    // this step's DMAs have landed; those of NST - 2 later steps may be in flight
    if (step + NST - 2 < nk) wait_vm_le<(NST - 2) * (WDMA + XDMA)>();
    else wait_vm_le<0>();
    block_sync();
    // refill the stage of the step before, which every wave has read
    if (step + NST - 1 < nk) issue(step + NST - 1);
    const char *ws = (const char *)s_t + (step % NST) * (BN + BM) * BK;
    const char *xs = ws + BN * BK;
#pragma unroll
    for (int c = 0; c < BK / 32; ++c) {
      i32x4 a[TI], b[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int nl = (wn * TI + i) * 32;
        if (MODE == 0) {
          const int row = nl + r32;
          a[i] = *(const i32x4 *)(ws + row * BK + 16 * swz(row, 2 * c + h));
        } else {
          // two transposing reads of 8 rows x 16 columns per 16 lanes
          const int t = (lane & 15) >> 1, ch = nl / 16 + ((lane >> 4) & 1);
          const int row = 32 * c + 16 * h + t;
          typedef __attribute__((address_space(3))) i32x2 lds2;
          const char *p = ws + row * BN + 16 * (ch ^ (row & 7)) + 8 * (lane & 1);
          const i32x2 lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)p);
          const i32x2 hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)(p + 8 * BN));
          a[i] = i32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int row = (wm * TJ + j) * 32 + r32;
        b[j] = *(const i32x4 *)(xs + row * BK + 16 * swz(row, 2 * c + h));
      }
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma_i8(a[i], b[j], acc[i][j]);
    }
  }

  // scales, then the rank-r term on the float32 values, rounded once to bf16
  float sx[TJ];
  int64_t mrow[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    mrow[j] = m0 + (wm * TJ + j) * 32 + r32;
    sx[j] = g.sx[mrow[j] < g.M ? mrow[j] : g.M - 1];
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int64_t nb = n0 + (wn * TI + i) * 32;
    f32x16 v[TJ];
    float4 sw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t n = nb + 8 * q + 4 * h;
      sw[q] = MODE == 0 ? *(const float4 *)(g.sw + (n < g.d ? n : g.d - 4))
                        : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float f = (float)acc[i][j][q] * sx[j];
        const float w[4] = {sw[q >> 2].x, sw[q >> 2].y, sw[q >> 2].z, sw[q >> 2].w};
        v[j][q] = MODE == 0 ? f * w[q & 3] : f;
      }
    for (int t0 = 0; t0 < g.rp; t0 += 16) {
      const int t = t0 + 8 * h;
      int64_t n = nb + r32;
      n = n < g.Ntot ? n : g.Ntot - 1;
      uint4 l;
      if (MODE == 0 && g.r % 8 == 0) {
        l = t < g.r ? *(const uint4 *)(g.L + n * g.r + t) : ql::zero4();
      } else {
        uint32_t e[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int tc = t + x < g.r ? t + x : g.r - 1;
          e[x] = g.L[MODE == 0 ? n * g.r + tc : tc * g.Ntot + n];
          e[x] = t + x < g.r ? e[x] : 0u;
        }
        l = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16),
                       e[6] | (e[7] << 16));
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int64_t m = mrow[j] < g.M ? mrow[j] : g.M - 1;
        const uint4 hi = *(const uint4 *)(g.Shi + m * g.rp + t);
        const uint4 lo = *(const uint4 *)(g.Slo + m * g.rp + t);
        v[j] = ql::mfma32(l, hi, v[j]);
        v[j] = ql::mfma32(l, lo, v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (mrow[j] >= g.M) continue;
      uint16_t *out = g.Out + mrow[j] * g.Ntot;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = nb + 8 * q + 4 * h;
        if (n < g.Ntot)
          *(uint2 *)(out + n) = make_uint2(ql::pack_bf16x2(v[j][4 * q], v[j][4 * q + 1]),
                                           ql::pack_bf16x2(v[j][4 * q + 2], v[j][4 * q + 3]));
      }
    }
  }
}

// ---- decode: up to 64 tokens ------------------------------------------------
// A workgroup of eight waves owns 16 rows of the weight and all tokens, its
// waves take 64-code chunks of the rows in turn (v_mfma_i32_16x16x64_i8: lane l
// supplies row l % 16, codes 16 (l / 16) .. +15 of both operands and holds
// rows 4 (l / 16) .. +3 of token l % 16); the waves' int32 sums meet in LDS.
// Bound by the weight's bytes: each is read once, in pieces of 512 consecutive
// bytes a row and round of waves.
struct I8Gemv {
  const int8_t *W;
  const float *sw;
  int64_t d, k;
  const int8_t *In;      // M x ldi
  int64_t ldi;
  const float *sx;
  int M;
  const uint16_t *B;     // d x r
  const float *H;        // M x rp
  int r, rp;
  float s;
  uint16_t *Y;           // M x d
};

constexpr int GV_W = 8;

template <int TB, int UN>
__global__ __launch_bounds__(64 * GV_W) void int8_gemv_kernel(I8Gemv g) {
  __shared__ int s_red[GV_W][TB][4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, grp = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t row = n0 + c16 < g.d ? n0 + c16 : g.d - 1;
  const int8_t *w = g.W + row * g.k + 16 * grp;
  const int8_t *x[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    const int m = 16 * b + c16 < g.M ? 16 * b + c16 : g.M - 1;
    x[b] = g.In + m * g.ldi + 16 * grp;
  }
  i32x4 acc[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) acc[b] = i32x4{0, 0, 0, 0};
  const int nc = (int)(g.k >> 6);
  for (int c = wave; c < nc; c += GV_W * UN) {
    i32x4 a[UN], v[UN][TB];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      // chunks past the end: the last one against zeros
      const int cc = c + u * GV_W, at = 64 * (cc < nc ? cc : nc - 1);
      a[u] = *(const i32x4 *)(w + at);
#pragma unroll
      for (int b = 0; b < TB; ++b) v[u][b] = *(const i32x4 *)(x[b] + at);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (c + u * GV_W >= nc) a[u] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < TB; ++b)
        acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], v[u][b], acc[b], 0, 0, 0);
    }
  }
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) s_red[wave][b][q][lane] = acc[b][q];
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * TB; o += 64 * GV_W) {
    const int n = o & 15, m = o >> 4, b = m >> 4;
    if (m >= g.M || n0 + n >= g.d) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < GV_W; ++v) sum += s_red[v][b][n & 3][16 * (n >> 2) + (m & 15)];
    float y = (float)sum * g.sx[m] * g.sw[n0 + n];
    if (g.r) {
      const uint16_t *bw = g.B + (n0 + n) * g.r;
      const float *hm = g.H + (int64_t)m * g.rp;
      float dot = 0.0f;
      for (int t = 0; t < g.r; ++t) dot = fmaf(hm[t], ql::bf16_to_f(bw[t]), dot);
      y += g.s * dot;
    }
    g.Y[(int64_t)m * g.d + n0 + n] = ql::f_to_bf16(y);
  }
}

}  // namespace

qlora_status launch_int8_gemm(int mode, const int8_t *W, const float *sw, int64_t d, int64_t k,
                              const int8_t *In, int64_t ldi, const float *sx, int64_t M,
                              const uint16_t *L, const uint16_t *hi, const uint16_t *lo, int r,
                              int rp, uint16_t *Out, hipStream_t st) {
  const I8Args g{W, sw, d, k, In, ldi, sx, M, mode == 0 ? d : k, mode == 0 ? k : d,
                 L, hi, lo, r, rp, Out};
  const unsigned grid = (unsigned)(ql_cdiv(g.Ntot, 128) * ql_cdiv(M, 256));
  QlProf prof(mode == 0 ? QLORA_K_INT8_GEMM_FWD : QLORA_K_INT8_GEMM_DX, st);
  if (mode == 0) int8_gemm_kernel<0, 128, 256, 2, 4, 3><<<grid, 512, 0, st>>>(g);
  else int8_gemm_kernel<1, 128, 256, 2, 4, 3><<<grid, 512, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

qlora_status launch_int8_gemv(const int8_t *W, const float *sw, int64_t d, int64_t k,
                              const int8_t *In, int64_t ldi, const float *sx, int64_t M,
                              const uint16_t *B, const float *H, int r, int rp, float s,
                              uint16_t *Y, hipStream_t st) {
  const I8Gemv g{W, sw, d, k, In, ldi, sx, (int)M, B, H, r, rp, s, Y};
  const unsigned grid = (unsigned)ql_cdiv(d, 16);
  QlProf prof(QLORA_K_INT8_GEMV, st);
  if (M <= 16) int8_gemv_kernel<1, 8><<<grid, 64 * GV_W, 0, st>>>(g);
  else if (M <= 32) int8_gemv_kernel<2, 4><<<grid, 64 * GV_W, 0, st>>>(g);
  else int8_gemv_kernel<4, 4><<<grid, 64 * GV_W, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}
