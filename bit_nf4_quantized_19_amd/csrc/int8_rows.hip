// Records of an 8-bit base and of the rows multiplied with it, gfx950.
//
// Row i of a bf16 matrix, optionally times one float32 factor per column
// (e = fl(x * mul), the gradient with the channel scales folded in):
//   s = fl(max|e| / 127),  q = clamp(rne(fl(e / s)), -127, 127),  s = 0: q = 0.
// One read of the row, which stays in registers between its maximum and its
// codes: a wave holds a row of up to 4096 values, a workgroup of four waves
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

// The code of e as the low byte of the result.
QL_DEV uint32_t code(float e, float inv, float s) {
  const float t = e * inv;
  const float b = t + kMagic;
  const float f = t - (b - kMagic);
  if (!(fabsf(f) < 0.5f - 0x1p-14f)) {   // near a half, or 1/s or t not finite
    float n = __builtin_rintf(__fdiv_rn(e, s));
    n = n < -127.0f ? -127.0f : n > 127.0f ? 127.0f : n;
    return n == n ? (uint32_t)(int)n & 255u : 0u;   // 0/0, inf/inf
  }
  return __float_as_uint(b);
}

QL_DEV uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
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

// WPR waves a row, chunks of 8 values; KEEP: CH chunks a lane hold the row.
template <int WPR, int CH, bool MUL, bool KEEP>
__global__ __launch_bounds__(256) void int8_rows_kernel(RowsArgs a) {
  __shared__ uint32_t s_max[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = WPR == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (row >= a.rows) return;   // WPR == 1 only: no barrier follows
  const int at = 8 * (WPR == 4 ? (int)threadIdx.x : lane);
  constexpr int STEP = 8 * 64 * WPR;
  const uint16_t *x = a.X + row * a.cols;
  uint4 v[CH];
  uint32_t top = 0;
  for (int c0 = 0; c0 < a.cols; c0 += CH * STEP) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      v[j] = col < a.cols ? *(const uint4 *)(x + col) : ql::zero4();
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      float e[8];
      values<MUL>(v[j], a.mul, col < a.cols ? col : 0, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // a lane past the end holds zeros; times a NaN factor they would not
        const uint32_t u = col < a.cols ? __float_as_uint(e[i]) & 0x7fffffffu : 0u;
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
    if (lane == 0) s_max[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = s_max[w] > top ? s_max[w] : top;
  }
  const float s = __fdiv_rn(__uint_as_float(top), 127.0f);
  const float inv = __fdiv_rn(1.0f, s);
  if (at == 0) a.scale[row] = s;
  int8_t *q = a.q + row * a.ldq;
  for (int c0 = 0; c0 < a.ldq; c0 += CH * STEP) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int col = c0 + j * STEP + at;
      if (col >= a.ldq) continue;
      uint2 out = make_uint2(0u, 0u);
      if (col < a.cols) {
        float e[8];
        const uint4 xv = KEEP ? v[j] : *(const uint4 *)(x + col);
        values<MUL>(xv, a.mul, col, e);
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = code(e[i], inv, s);
        out = make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
      }
      *(uint2 *)(q + col) = out;
    }
    if (KEEP) break;
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
