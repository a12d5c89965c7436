// Records of an 8-bit base and of the rows multiplied with it, gfx950.
//
// Row i of a bf16 matrix, optionally times one float32 factor per column
// (e = fl(x * mul), the gradient with the channel scales folded in):
//   s = fl(max|e| / 127),  q = clamp(rne(fl(e / s)), -127, 127),  s = 0: q = 0.
// One read of the row, which stays in registers between its maximum and its
// codes: a wave holds a row of up to 1024 values, a workgroup of four waves
// one of up to 16384; longer rows are read a second time. HBM-bound: 2 bytes
// read and 1 written per value.
//
// The maximum is taken over the bit patterns without their sign, where a NaN
// is above infinity, so a row that holds either gets that as its scale and
// its products become NaN. The quotient is formed as x * (1/s), which is off
// by less than 2^-15 for |x/s| <= 127 (1/s and the product each within 2^-23
// relative); only where that leaves the whole number open, within 2^-14 of a
// half, is the correctly rounded division taken.
#include "kernels.h"

namespace {

struct RowsArgs {
  const uint16_t *X;   // rows x cols
  int64_t rows;
  int cols;            // a multiple of 8
  const float *mul;    // [cols] (MUL) or unused
  int8_t *q;           // rows x ldq, zero past cols
  int ldq;             // a multiple of 8
  float *scale;        // [rows]
};

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number

// A row's scale and how its values become codes.
struct RowScale {
  float s, inv;
  bool plain;   // 1/s and every value / s are finite and far from the denormals
};
QL_DEV RowScale row_scale(uint32_t top) {
  RowScale r;
  r.s = __fdiv_rn(__uint_as_float(top), 127.0f);
  r.inv = __fdiv_rn(1.0f, r.s);
  r.plain = r.s >= 0x1p-120f && r.s <= 0x1p120f;
  return r;
}

QL_DEV uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}

// Eight codes. The quotients' check is one branch for all eight: a branch a
// value cost more than the arithmetic (2048 x 4096: 7.3 us).
QL_DEV uint2 codes8(const float (&e)[8], const RowScale &r) {
  uint32_t c[8];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = e[i] * r.inv, b = t + kMagic;
    far = fmaxf(far, fabsf(t - (b - kMagic)));
    c[i] = __float_as_uint(b);
  }
  if (!r.plain || far >= 0.5f - 0x1p-14f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float n = __builtin_rintf(__fdiv_rn(e[i], r.s));
      n = n < -127.0f ? -127.0f : n > 127.0f ? 127.0f : n;
      c[i] = n == n ? (uint32_t)(int)n : 0u;   // 0/0, inf/inf
    }
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

template <bool MUL>
QL_DEV void values(const uint4 &x, const float *mul, int col, float (&e)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[2 * i] = ql::bf16lo(w[i]);
    e[2 * i + 1] = ql::bf16hi(w[i]);
  }
  if (MUL) {
    const float4 a = *(const float4 *)(mul + col), b = *(const float4 *)(mul + col + 4);
    const float m[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __fmul_rn(e[i], m[i]);
  }
}

// One row by WPR waves, `at` this thread's first value; chunks of 8 values.
// KEEP: CH chunks a thread hold the row. With WPR == 4 the workgroup's threads
// come here together (s_max: four words of this row's waves).
template <int WPR, int CH, bool MUL, bool KEEP>
QL_DEV void row_record(const RowsArgs &a, int64_t row, int at, uint32_t *s_max) {
  const bool live = row < a.rows;
  constexpr int STEP = 8 * 64 * WPR;
  const uint16_t *x = a.X + (live ? row : 0) * a.cols;
  const int cols = live ? a.cols : 0;
  uint4 v[CH];
  uint32_t top = 0;
  for (int c0 = 0; c0 < a.cols; c0 += CH * STEP) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      v[j] = col < cols ? *(const uint4 *)(x + col) : ql::zero4();
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      if (c0 + j * STEP >= a.cols) break;
      float e[8];
      values<MUL>(v[j], a.mul, col < cols ? col : 0, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // a lane past the end holds zeros; times a NaN factor they would not
        const uint32_t u = col < cols ? __float_as_uint(e[i]) & 0x7fffffffu : 0u;
        top = u > top ? u : top;
      }
    }
    if (KEEP) break;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint32_t u = __shfl_xor(top, o);
    top = u > top ? u : top;
  }
  if (WPR == 4) {
    if ((threadIdx.x & 63) == 0) s_max[(threadIdx.x >> 6) & 3] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = s_max[w] > top ? s_max[w] : top;
  }
  if (!live) return;
  const RowScale rs = row_scale(top);
  if (at == 0) a.scale[row] = rs.s;
  int8_t *q = a.q + row * a.ldq;
  for (int c0 = 0; c0 < a.ldq; c0 += CH * STEP) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      if (col >= a.ldq) continue;
      uint2 out = make_uint2(0u, 0u);
      if (col < cols) {
        float e[8];
        const uint4 xv = KEEP ? v[j] : *(const uint4 *)(x + col);
        values<MUL>(xv, a.mul, col, e);
        out = codes8(e, rs);
      }
      *(uint2 *)(q + col) = out;
    }
    if (KEEP) break;
  }
}

template <int WPR, int CH, bool MUL, bool KEEP>
__global__ __launch_bounds__(256) void int8_rows_kernel(RowsArgs a) {
  __shared__ uint32_t s_max[4];
  const int64_t row = WPR == 4 ? (int64_t)blockIdx.x
                               : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  row_record<WPR, CH, MUL, KEEP>(a, row, 8 * (int)(threadIdx.x & (64 * WPR - 1)), s_max);
}

// ---- a linear's first launch: the tokens' records and the rank-r products -------
// out[m][t] = sum_c In[m][c] P[t][c] beside the records: a workgroup holds four
// rows in registers, so In is read once, and every four ranks of P meet them in
// 4x4x4 products of 16 blocks: lane l holds row l % 4 (of In, and of P) and 8
// columns of block l / 4, so that a load takes 256 consecutive bytes of four
// rows. The 16 blocks' sums are taken by exchanges that halve the sums a lane
// holds with the lanes a sum is spread over; the waves' sums meet in LDS in
// order. 2048 x 4096, r = 16: 14 us; the records and the products one after the
// other 15, with 16x16 products (16 rows x 64 bytes a load, which the address
// units take twice as long for) 17, with two-element dot products (a quarter of
// the rate of other vector instructions) 15. Sixteen more ranks add 4 us: P is
// read by every workgroup, from L2. 16 tokens: 6 us against 10.
struct PrepArgs {
  RowsArgs rows;       // rows.q == NULL: no records
  const uint16_t *P;   // pr x cols; rows past pr count as zeros
  int pr, rp, r;
  int per;             // ranks of a workgroup, a multiple of NR
  float *out, *out2;   // M x rp, M x r (out2 may be NULL)
  // M x rp: s out as bf16 high and low parts, 2^-16 of it at most left out: two
  // bf16 products for it in the GEMM's epilogue, whose output is rounded to 2^-8
  uint16_t *hi, *lo;
  float s;
  int *zero;           // nzero ints cleared, for a later launch of the call
  int64_t nzero;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
// D[i][j] of block l / 4 += sum over 4 columns: lane l supplies row l % 4 of both
// operands and holds D[0 .. 3][l % 4].
QL_DEV f32x4 mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, const f32x4 &c) {
  const uint2 a = make_uint2(a0, a1), b = make_uint2(b0, b1);
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, a),
                                                __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// lane ^ 8 (rotation by 8 of a row of 16) and lane ^ 4 (^ 7, then ^ 3)
QL_DEV float lane8(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xf, 0xf, true));
}
QL_DEV float lane4(float v) {
  const int x = __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xf, 0xf, true);
  return __int_as_float(__builtin_amdgcn_mov_dpp(x, 0x1B, 0xf, 0xf, true));
}
// Sums over the 16 blocks of N (16 or 4) values a lane: lane l ends with value
// (l / 4) % N of its l % 4 in v[0].
template <int N>
QL_DEV void block_sums(float (&v)[N], int lane) {
#pragma unroll
  for (int i = 0; i < (N == 16 ? 8 : N); ++i) {
    const uint32_t x = __float_as_uint(v[i]), y = __float_as_uint(v[N == 16 ? i + 8 : i]);
    const u32x2 z =
        __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, y, false, false));
    v[i] = __uint_as_float(z[0]) + __uint_as_float(z[1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __float_as_uint(v[i]), y = __float_as_uint(v[N == 16 ? i + 4 : i]);
    const u32x2 z =
        __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, y, false, false));
    v[i] = __uint_as_float(z[0]) + __uint_as_float(z[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 8 ? v[i + 2] : v[i], give = lane & 8 ? v[i] : v[i + 2];
    v[i] = keep + lane8(give);
  }
  const float keep = lane & 4 ? v[1] : v[0], give = lane & 4 ? v[0] : v[1];
  v[0] = keep + lane4(give);
}

// RG groups of four rows, NW waves, CH chunks of 128 columns each; NR ranks (16
// or 4) at a time, their fours in an order that differs between workgroups.
template <int RG, int NW, int CH, int NR, bool MUL>
__global__ __launch_bounds__(64 * NW) void int8_prep_kernel(PrepArgs a) {
  __shared__ uint32_t s_max[NW][4 * RG];
  __shared__ float s_sum[NW][4 * NR * RG];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, j4 = lane & 3;
  const int cols = a.rows.cols;
  const int64_t row0 = (int64_t)blockIdx.x * 4 * RG + j4, rows = a.rows.rows;
  for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 * NW + tid; i < a.nzero;
       i += (int64_t)gridDim.x * gridDim.y * 64 * NW)
    a.zero[i] = 0;
  const int at = 128 * wave + 8 * (lane >> 2);   // column of chunk 0
  constexpr int STEP = 128 * NW;
  uint4 v[RG][CH];
#pragma unroll
  for (int y = 0; y < RG; ++y)
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = j * STEP + at;
      v[y][j] = col < cols && row0 + 4 * y < rows
                    ? *(const uint4 *)(a.rows.X + (row0 + 4 * y) * cols + col) : ql::zero4();
    }
  const int begin = (int)blockIdx.y * a.per;
  const int end = begin + a.per < a.rp ? begin + a.per : a.rp;
  constexpr int NG = NR / 4;
  const int rot = (int)blockIdx.x & (NG - 1);
  constexpr int PD = NG > 1 ? 2 : 1;   // groups of P in registers (4: no faster)
  uint4 p[PD][CH];
  auto ranks = [&](int buf, int t) {   // ranks t .. t + 3 of P
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = j * STEP + at;
      p[buf][j] = col < cols && t + j4 < a.pr
                      ? *(const uint4 *)(a.P + (int64_t)(t + j4) * cols + col) : ql::zero4();
    }
  };
#pragma unroll
  for (int g = 0; g < (PD > 1 ? PD - 1 : 1); ++g)   // under the records
    ranks(g, begin + 4 * ((g + rot) & (NG - 1)));
  if (a.rows.q && blockIdx.y == 0) {
#pragma unroll
    for (int y = 0; y < RG; ++y) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int col = j * STEP + at;
        if (j * STEP >= cols) break;
        float e[8];
        values<MUL>(v[y][j], a.rows.mul, col < cols ? col : 0, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // a lane past the end holds zeros; times a NaN factor they would not
          const uint32_t u = col < cols ? __float_as_uint(e[i]) & 0x7fffffffu : 0u;
          top = u > top ? u : top;
        }
      }
#pragma unroll
      for (int o = 32; o >= 4; o >>= 1) {
        const uint32_t u = __shfl_xor(top, o);
        top = u > top ? u : top;
      }
      if (lane < 4) s_max[wave][4 * y + lane] = top;
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < RG; ++y) {
      const int64_t row = row0 + 4 * y;
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = s_max[w][4 * y + j4] > top ? s_max[w][4 * y + j4] : top;
      const RowScale rs = row_scale(top);
      if (row >= rows) continue;
      if (tid < 4) a.rows.scale[row] = rs.s;
      int8_t *q = a.rows.q + row * a.rows.ldq;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int col = j * STEP + at;
        if (col >= a.rows.ldq) continue;
        uint2 out = make_uint2(0u, 0u);
        if (col < cols) {
          float e[8];
          values<MUL>(v[y][j], a.rows.mul, col, e);
          out = codes8(e, rs);
        }
        *(uint2 *)(q + col) = out;
      }
    }
  }
  for (int t0 = begin; t0 < end; t0 += NR) {
    float acc[RG][NR];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int buf = g % PD, h = g + PD - 1;   // h: the group PD - 1 ahead
      const int next = t0 + NR * (h / NG) + 4 * ((h + rot) & (NG - 1));
      if (PD > 1 && next < end) ranks(h % PD, next);
#pragma unroll
      for (int y = 0; y < RG; ++y) {
        f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f}, d2 = d;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          d = mfma4(p[buf][j].x, p[buf][j].y, v[y][j].x, v[y][j].y, d);
          d2 = mfma4(p[buf][j].z, p[buf][j].w, v[y][j].z, v[y][j].w, d2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[y][4 * g + i] = d[i] + d2[i];
      }
      __builtin_amdgcn_sched_barrier(0);   // loads stay PD - 1 groups ahead, not more
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < RG; ++y) {
      block_sums<NR>(acc[y], lane);
      if (lane < 4 * NR) s_sum[wave][4 * NR * y + lane] = acc[y][0];
    }
    __syncthreads();
    for (int o = tid; o < 4 * NR * RG; o += 64 * NW) {   // row o % 4 of group y, value x
      const int y = o / (4 * NR), x = (o >> 2) & (NR - 1);
      const int64_t row = (int64_t)blockIdx.x * 4 * RG + 4 * y + (o & 3);
      const int t = t0 + (NG > 1 ? 4 * (((x >> 2) + rot) & (NG - 1)) + (x & 3) : x);
      if (row >= rows) continue;
      float h = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) h += s_sum[w][o];
      a.out[row * a.rp + t] = h;
      if (a.out2 && t < a.r) a.out2[row * a.r + t] = h;
      if (a.hi) {
        const float f = a.s * h;
        const uint16_t up = ql::f_to_bf16(f);
        a.hi[row * a.rp + t] = up;
        a.lo[row * a.rp + t] = ql::f_to_bf16(f - ql::bf16_to_f(up));
      }
    }
  }
}

// ---- a backward's copies ----------------------------------------------------------
struct CopyArgs {
  const uint16_t *A, *B;
  int64_t d, k, M;
  int r, rp;
  uint16_t *At, *Bt;
  const float *H;
  float *Hp;
};
// A thread takes eight ranks (grid row y) of one row of B, written as a column
// of Bt, of one column of A, or of one row of H; neighbours' are consecutive.
__global__ __launch_bounds__(256) void int8_layout_kernel(CopyArgs a) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t0 = 8 * (int)blockIdx.y;
  uint32_t e[8];
  if (i < a.d) {
    const uint16_t *b = a.B + i * a.r;
    if (a.r % 8 == 0) {
      const uint4 v = t0 < a.r ? *(const uint4 *)(b + t0) : ql::zero4();
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int x = 0; x < 8; ++x) e[x] = w[x >> 1] >> (16 * (x & 1));
    } else {
#pragma unroll
      for (int x = 0; x < 8; ++x) e[x] = t0 + x < a.r ? b[t0 + x] : 0u;
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) a.Bt[(t0 + x) * a.d + i] = (uint16_t)e[x];
    return;
  }
  i -= ql_rup(a.d, 256);
  if (i < 0) return;
  if (i < a.k) {
#pragma unroll
    for (int x = 0; x < 8; ++x) e[x] = t0 + x < a.r ? a.A[(t0 + x) * a.k + i] : 0u;
    *(uint4 *)(a.At + i * a.rp + t0) = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16),
                                                  e[4] | (e[5] << 16), e[6] | (e[7] << 16));
    return;
  }
  i -= ql_rup(a.k, 256);
  if (a.H && i >= 0 && i < a.M) {
    float h[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) h[x] = t0 + x < a.r ? a.H[i * a.r + t0 + x] : 0.0f;
    *(float4 *)(a.Hp + i * a.rp + t0) = make_float4(h[0], h[1], h[2], h[3]);
    *(float4 *)(a.Hp + i * a.rp + t0 + 4) = make_float4(h[4], h[5], h[6], h[7]);
  }
}

template <bool MUL>
void launch(const RowsArgs &a, hipStream_t st) {
  const int n = a.ldq;
  const unsigned four = (unsigned)ql_cdiv(a.rows, 4), one = (unsigned)a.rows;
  if (n <= 1024) int8_rows_kernel<1, 2, MUL, true><<<four, 256, 0, st>>>(a);
  else if (n <= 4096) int8_rows_kernel<4, 2, MUL, true><<<one, 256, 0, st>>>(a);
  else if (n <= 8192) int8_rows_kernel<4, 4, MUL, true><<<one, 256, 0, st>>>(a);
  else if (n <= 16384) int8_rows_kernel<4, 8, MUL, true><<<one, 256, 0, st>>>(a);
  else int8_rows_kernel<4, 4, MUL, false><<<one, 256, 0, st>>>(a);
}

}  // namespace

qlora_status launch_int8_rows(const uint16_t *X, int64_t rows, int64_t cols, const float *mul,
                              int8_t *q, int64_t ldq, float *scale, hipStream_t st) {
  const RowsArgs a{X, rows, (int)cols, mul, q, (int)ldq, scale};
  QlProf prof(QLORA_K_INT8_ROWS, st);
  if (mul) launch<true>(a, st);
  else launch<false>(a, st);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

qlora_status launch_int8_layout(const uint16_t *A, const uint16_t *B, int64_t d, int64_t k, int r,
                                int rp, uint16_t *At, uint16_t *Bt, const float *H, int64_t M,
                                float *Hp, hipStream_t st) {
  const CopyArgs a{A, B, d, k, M, r, rp, At, Bt, H, Hp};
  const int64_t n = ql_rup(d, 256) + ql_rup(k, 256) + (H ? M : 0);
  QlProf prof(QLORA_K_LAYOUT, st);
  int8_layout_kernel<<<dim3((unsigned)ql_cdiv(n, 256), (unsigned)(rp / 8)), 256, 0, st>>>(a);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

qlora_status launch_int8_prep(const uint16_t *X, int64_t rows, int64_t cols, const float *mul,
                              int8_t *q, int64_t ldq, float *scale, const Int8Rank &k,
                              hipStream_t st) {
  // many rows: eight a workgroup, which halves the reads of P; few: their ranks
  // by fours over more workgroups, which read In again
  const bool many = rows >= 1024, few = rows <= 256;
  if (cols > 16384 || (cols > 8192 && !few)) {   // past a workgroup's registers: two launches
    const qlora_status s =
        q ? launch_int8_rows(X, rows, cols, mul, q, ldq, scale, st) : QLORA_OK;
    if (s != QLORA_OK) return s;
    return launch_skinny(X, rows, cols, k.P, false, k.pr, k.rp, k.out, k.out2, k.r, k.s, k.hi,
                         k.lo, st, k.zero, k.nzero);
  }
  const PrepArgs a{{X, rows, (int)cols, mul, q, (int)ldq, scale}, k.P, k.pr, k.rp, k.r,
                   few ? 4 : k.rp, k.out, k.out2, k.hi, k.lo, k.s, k.zero, k.nzero};
  const dim3 grid((unsigned)ql_cdiv(rows, many ? 8 : 4), (unsigned)(few ? k.rp / 4 : 1));
  QlProf prof(QLORA_K_INT8_ROWS, st);
#define QL_PREP(RG, NW, C, N)                                                      \
  if (mul) int8_prep_kernel<RG, NW, C, N, true><<<grid, 64 * NW, 0, st>>>(a);      \
  else int8_prep_kernel<RG, NW, C, N, false><<<grid, 64 * NW, 0, st>>>(a);
  if (cols <= 4096) {
    if (few) { QL_PREP(1, 8, 4, 4) }
    else if (many) { QL_PREP(2, 8, 4, 16) }
    else { QL_PREP(1, 8, 4, 16) }
  } else if (cols <= 8192) {
    if (few) { QL_PREP(1, 8, 8, 4) }
    else if (many) { QL_PREP(2, 8, 8, 16) }
    else { QL_PREP(1, 8, 8, 16) }
  } else {
    QL_PREP(1, 16, 8, 4)
  }
#undef QL_PREP
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}
