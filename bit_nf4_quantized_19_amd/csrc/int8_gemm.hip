// Integer GEMM and decode product of the 8-bit base with the LoRA rank-r
// term, gfx950 MFMA.
//
//   forward: Y[m][n]  = sx[m] sw[n] sum_K Wq[n][K] Xq[m][K] + sum_t B[n][t] (sH)[m][t]
//   dX:      dX[m][n] = se[m] sum_K Wq[K][n] Eq[m][K]       + sum_t A[t][n] (sG)[m][t]
//
// The integer sums are exact in int32 (K <= 131072), so how they are split
// does not change a bit of the result. As in the NF4 GEMM the product is
// computed transposed (weights are the MFMA's A operand), so each lane ends
// with 4 consecutive n of one token, and s H (s G) comes as bf16 hi + lo parts
// (together to 2^-16 of each value, before the output's rounding to 2^-8).
//
// GEMM: tile 128 (n) x 256 (m), K-step 128, eight waves of 32 x 128, one
// workgroup per CU. Both tiles' rows of a step (384 x 128 bytes) come by LDS DMA,
// three stages, two to three steps ahead; in a step every wave reads the operands
// of a K-slice of 64 while the products of the slice before run, and the one
// barrier of the step lies between its two slices, so that the first reads of
// the next stage run under the second slice's products. dX needs the weight's
// columns: its tile holds 128 rows of the weight as they lie in memory, read by
// the transposing LDS read (8 rows x 16 columns per 16 lanes). LDS rows are
// permuted by 16-byte chunks (no bank conflicts counted in either mode).
// 2048 tokens of 4096 x 4096: forward 37-40 us (1.7-1.85 POP/s; the vendor
// library's int8 product of that shape, without scales and rank-r term, 42), dX
// 38-41. A step takes 0.82-0.97 us for 0.43 of matrix work at the full clock.
// L2 serves 81% of the requests (85 MB of misses).
#include "kernels.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

struct I8Args {
  const int8_t *W;       // d x k codes
  const float *sw;       // [d]
  int64_t d, k;
  const int8_t *In;      // M x ldi codes, zero past Ktot
  int64_t ldi;           // a multiple of 128
  const float *sx;       // [M]
  int64_t M, Ntot, Ktot;
  const uint16_t *L;     // rank-r term: Ntot x ldl, zero past r where ldl > r
  int ldl;
  const uint16_t *Shi, *Slo;   // M x rp
  int rp;
  uint16_t *Out;         // M x Ntot
  int S;                 // workgroups that share a tile's K-steps
  i32x4 *part;           // S > 1: their sums, [split][tile][block][thread]
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

// 16x16x64: lane l supplies row l % 16, codes 16 (l / 16) .. +15 of both
// operands and holds rows 4 (l / 16) .. +3 of column l % 16. The 32x32x32 form
// has the same rate but draws more power, and the chip is power-limited here:
// 4.0 against 3.4 POP/s sustained on random codes.
QL_DEV i32x4 mfma_i8(const i32x4 &a, const i32x4 &b, const i32x4 &c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A token's scale as two factors, (s, 1) or, from 2^96 on, (s 2^-64, 2^64): a sum
// (below 2^31) times the first does not overflow, so that a small channel scale
// still makes it the ordinary number that it is before the second is taken.
QL_DEV float2 token_scale(float s) {
  return s > 0x1p96f ? make_float2(s * 0x1p-64f, 0x1p64f) : make_float2(s, 1.0f);
}

constexpr int BK = 128;   // K-step: 128 codes
constexpr int SL = BK / 64;   // K-slices of a step

// Where chunk (16 bytes) c of a tile row is kept in its row, so that what one
// operand read takes lies in different banks (64 of 4 bytes). K-contiguous
// tiles have rows of 128 bytes and are read 16 rows x 16 bytes at a time;
// the weight tile of dX has rows of BN bytes and is read 8 rows x 16 columns
// at a time, from two groups of 8 rows 16 apart.
QL_DEV int swz(int row, int c) { return c ^ ((row >> 1) & 7); }
QL_DEV int swz_dx(int row, int c) { return c ^ (row & 7) ^ ((row >> 4) & 1); }

// First column and token of tile id. XCD-aware order: workgroups of one XCD
// (id % 8) take a contiguous range, in groups of 4 token blocks with the column
// tile slow, so that an XCD's L2 serves its 32 tiles' shared rows.
template <int BN, int BM>
QL_DEV void tile_of(const I8Args &g, uint32_t bid, int64_t &n0, int64_t &m0) {
  const uint32_t tn = (uint32_t)((g.Ntot + BN - 1) / BN), tm = (uint32_t)((g.M + BM - 1) / BM);
  const uint32_t nt = tn * tm, q = nt / 8, rest = nt % 8, x = bid % 8;
  const uint32_t id = x * q + (x < rest ? x : rest) + bid / 8;
  const uint32_t g0 = id / (4 * tn) * 4, gm = tm - g0 < 4 ? tm - g0 : 4, in = id - g0 * tn;
  n0 = (int64_t)(in / gm) * BN;
  m0 = (int64_t)(g0 + in % gm) * BM;
}

// What the epilogue of a wave's 16 TI x 16 TJ block at column n0, token m0 reads:
// scales and the operands of 16 ranks, loaded under the last products. Lanes
// 0-31 take s H's high parts, lanes 32-63 its low parts, against the same rows
// of L.
template <int MODE, int TI, int TJ>
struct EpilogueIn {
  float sx[TJ];
  float4 sw[TI];
  uint4 l[2][TI], s[2][TJ];   // ranks t0 .. t0 + 15 in buffer t0 / 16 % 2

  QL_DEV void ranks(const I8Args &g, int64_t n0, int64_t m0, int t0, int b) {
    const int lane = threadIdx.x & 63, c16 = lane & 15, grp = lane >> 4, t = t0 + 8 * (grp & 1);
    const uint16_t *S = grp < 2 ? g.Shi : g.Slo;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t m = m0 + 16 * j + c16;
      s[b][j] = *(const uint4 *)(S + (m < g.M ? m : g.M - 1) * g.rp + t);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      int64_t n = n0 + 16 * i + c16;
      n = n < g.Ntot ? n : g.Ntot - 1;
      if (g.ldl % 8 == 0) {
        l[b][i] = t < g.ldl ? *(const uint4 *)(g.L + n * g.ldl + t) : ql::zero4();
      } else {
        uint32_t e[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int tc = t + x < g.ldl ? t + x : g.ldl - 1;
          e[x] = g.L[n * g.ldl + tc];
          e[x] = t + x < g.ldl ? e[x] : 0u;
        }
        l[b][i] = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16),
                             e[6] | (e[7] << 16));
      }
    }
  }
  QL_DEV void load(const I8Args &g, int64_t n0, int64_t m0) {
    const int lane = threadIdx.x & 63, c16 = lane & 15, grp = lane >> 4;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t m = m0 + 16 * j + c16;
      sx[j] = g.sx[m < g.M ? m : g.M - 1];
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t n = n0 + 16 * i + 4 * grp;
      sw[i] = MODE == 0 ? *(const float4 *)(g.sw + (n < g.d ? n : g.d - 4))
                        : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    }
    if (g.rp) ranks(g, n0, m0, 0, 0);
  }
};

// The block's scales, then the rank-r term on the float32 values, rounded once
// to bf16. The block goes through the wave's TI * TJ * 512 bytes of LDS, so
// that whole lines of 128 bytes are stored: 8-byte stores of the lanes' four
// columns took 7 us more for 2048 x 4096 outputs.
template <int MODE, int TI, int TJ>
QL_DEV void epilogue(const I8Args &g, const i32x4 (&acc)[TI][TJ], EpilogueIn<MODE, TI, TJ> &in,
                     char *blk, int64_t n0, int64_t m0) {
  const int lane = threadIdx.x & 63, c16 = lane & 15, grp = lane >> 4;
  constexpr int WB = TI * 32, CPW = WB / 16;   // bytes and chunks of a block's row
  static_assert((CPW & (CPW - 1)) == 0, "a power of two");
  if (g.rp > 16) in.ranks(g, n0, m0, 16, 1);
  f32x4 v[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const float w[4] = {in.sw[i].x, in.sw[i].y, in.sw[i].z, in.sw[i].w};
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const float2 s = token_scale(in.sx[j]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float f = (float)acc[i][j][q];
        v[i][j][q] = MODE == 0 ? f * s.x * w[q] * s.y : f * in.sx[j];
      }
    }
  }
  for (int t0 = 0; t0 < g.rp; t0 += 32)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (t0 + 16 * h >= g.rp) break;
      uint4 l[TI], sv[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) l[i] = in.l[h][i];
#pragma unroll
      for (int j = 0; j < TJ; ++j) sv[j] = in.s[h][j];
      if (t0 + 16 * h + 32 < g.rp) in.ranks(g, n0, m0, t0 + 16 * h + 32, h);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) v[i][j] = ql::mfma16(l[i], sv[j], v[i][j]);
    }
  // row j * 16 + c16 of the block, columns 16 i + 4 grp .. +3, the row's 16-byte
  // chunks permuted by the row
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int row = 16 * j + c16, c = (2 * i + (grp >> 1)) ^ (c16 & (CPW - 1));
      *(uint2 *)(blk + row * WB + 16 * c + 8 * (grp & 1)) =
          make_uint2(ql::pack_bf16x2(v[i][j][0], v[i][j][1]),
                     ql::pack_bf16x2(v[i][j][2], v[i][j][3]));
    }
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int x = 0; x < TJ * 16 * CPW / 64; ++x) {
    const int row = x * (64 / CPW) + lane / CPW, c = lane % CPW;
    const uint4 o = *(const uint4 *)(blk + row * WB + 16 * (c ^ (row & 15 & (CPW - 1))));
    const int64_t m = m0 + row, n = n0 + 8 * c;
    if (m < g.M && n < g.Ntot) *(uint4 *)(g.Out + m * g.Ntot + n) = o;
  }
}

// MODE 0 forward, 1 dX. BN x BM tile by WN x WM waves, NST LDS stages; SPLIT:
// g.S workgroups share the tile's K-steps and leave their sums in g.part.
template <int MODE, int BN, int BM, int WN, int WM, int NST, bool SPLIT>
__global__ __launch_bounds__(64 * WN * WM) void int8_gemm_kernel(I8Args g) {
  constexpr int NW = WN * WM, TI = BN / WN / 16, TJ = BM / WM / 16;
  constexpr int WDMA = BN * BK / 1024 / NW, XDMA = BM * BK / 1024 / NW;
  constexpr uint32_t STAGE = (BN + BM) * BK;
  __shared__ __align__(1024) uint4 s_t[NST * STAGE / 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN, c16 = lane & 15, grp = lane >> 4;
  uint32_t tile = blockIdx.x;
  int first = 0, nk = (int)ql_cdiv(g.Ktot, BK);   // this workgroup's K-steps
  if (SPLIT) {
    // tile fast: an XCD's workgroups share tokens of one range of K
    const uint32_t nt = gridDim.x / (uint32_t)g.S, y = tile / nt;
    tile -= y * nt;
    first = (int)(y * (uint32_t)nk / (uint32_t)g.S);
    nk = (int)((y + 1) * (uint32_t)nk / (uint32_t)g.S) - first;
  }
  int64_t n0, m0;
  tile_of<BN, BM>(g, tile, n0, m0);

  // this lane's DMA sources (rows and columns past the matrix fetch the last
  // valid ones: their sums are not stored, or meet the zeros of In past Ktot)
  const int8_t *xsrc[XDMA], *wsrc[WDMA];
  uint32_t wrow[WDMA];   // forward: offset in the row's step; dX: row of the step
#pragma unroll
  for (int i = 0; i < XDMA; ++i) {
    const int row = 8 * (XDMA * wave + i) + (lane >> 3);
    const int64_t m = m0 + row < g.M ? m0 + row : g.M - 1;
    xsrc[i] = g.In + m * g.ldi + 16 * swz(row, lane & 7);
  }
#pragma unroll
  for (int i = 0; i < WDMA; ++i) {
    if (MODE == 0) {
      const int row = 8 * (WDMA * wave + i) + (lane >> 3);
      const int64_t n = n0 + row < g.d ? n0 + row : g.d - 1;
      wrow[i] = 16 * swz(row, lane & 7);
      wsrc[i] = g.W + n * g.k;
    } else {
      constexpr int CPR = BN / 16;   // chunks of a tile row
      const int p = 64 * (WDMA * wave + i) + lane;
      wrow[i] = p / CPR;
      const int64_t n = n0 + 16 * swz_dx(wrow[i], p % CPR);
      wsrc[i] = g.W + (n < g.k ? n : g.k - 16);
    }
  }
  const uint32_t k = (uint32_t)g.k, wend = MODE == 0 ? k - 16 : (uint32_t)g.d - 1;
  auto issue = [&](int step, uint32_t stage) {   // stage: its byte offset
    const uint32_t kk = (uint32_t)(first + step) * BK, base = lds_addr(s_t) + stage;
#pragma unroll
    for (int i = 0; i < WDMA; ++i) {
      const uint32_t e = kk + wrow[i] < wend ? kk + wrow[i] : wend;
      dma16(wsrc[i] + (MODE == 0 ? (uint64_t)e : (uint64_t)e * k), base + 1024 * (WDMA * wave + i));
    }
#pragma unroll
    for (int i = 0; i < XDMA; ++i)
      dma16(xsrc[i] + kk, base + BN * BK + 1024 * (XDMA * wave + i));
  };

  // LDS offsets of this lane's operands: the K-contiguous ones by K-slice
  // (rows 16 apart are permuted alike), those of a dX weight tile by block
  uint32_t koff[SL], noff[TI];
#pragma unroll
  for (int c = 0; c < SL; ++c) koff[c] = c16 * BK + 16 * swz(c16, 4 * c + grp);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int row = 16 * grp + (c16 >> 1);
    noff[i] = row * BN + 16 * swz_dx(row, wn * TI + i) + 8 * (lane & 1);
  }

  i32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // operands of a K-slice and of the slice after it, read under its products
  i32x4 fa[2][TI], fb[2][TJ];
  auto read = [&](uint32_t stage, int c) {
    const char *ws = (const char *)s_t + stage, *xs = ws + BN * BK;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      if (MODE == 0) {
        fa[c][i] = *(const i32x4 *)(ws + koff[c] + (wn * TI + i) * 16 * BK);
      } else {
        // two transposing reads, each 8 rows x 16 columns per 16 lanes: lane
        // 2 t + e addresses columns 8 e .. +7 of row t and gets the 8 rows of
        // column lane % 16 (rows 8 on are permuted like rows 0 on)
        typedef __attribute__((address_space(3))) i32x2 lds2;
        const char *q = ws + noff[i] + 64 * c * BN;
        const i32x2 lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)q);
        const i32x2 hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)(q + 8 * BN));
        fa[c][i] = i32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      fb[c][j] = *(const i32x4 *)(xs + koff[c] + (wm * TJ + j) * 16 * BK);
  };
  auto products = [&](int c, int i0, int i1) {
#pragma unroll
    for (int i = i0; i < i1; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = mfma_i8(fa[c][i], fb[c][j], acc[i][j]);
  };
  static_assert(SL == 2, "two slices a step, one operand set each");

  for (int s = 0; s < NST && s < nk; ++s) issue(s, s * STAGE);
  // step 0's DMAs have landed; those of NST - 1 later steps may be in flight
  if (NST <= nk) wait_vm_le<(NST - 1) * (WDMA + XDMA)>();
  else wait_vm_le<0>();
  block_sync();
  read(0, 0);
  uint32_t stage = 0;
  for (int step = 0; step + 1 < nk; ++step) {
    read(stage, 1);
    products(0, 0, TI);
    // this wave has read its stage whole, and so has every wave past the
    // barrier: the stage is refilled. The next one is ready once its DMAs have
    // landed (those of NST - 2 later steps may be in flight)
    if (step + NST - 1 < nk) wait_vm_le<(NST - 2) * (WDMA + XDMA)>();
    else wait_vm_le<0>();
    block_sync();
    const uint32_t next = stage + STAGE == NST * STAGE ? 0 : stage + STAGE;
    read(next, 0);
    products(1, 0, 1);
    if (step + NST < nk) issue(step + NST, stage);
    products(1, 1, TI);
    stage = next;
  }
  read(stage, 1);
  EpilogueIn<MODE, TI, TJ> in;
  if (!SPLIT) in.load(g, n0 + wn * TI * 16, m0 + wm * TJ * 16);
  products(0, 0, TI);
  products(1, 0, TI);

  if (SPLIT) {
    i32x4 *to = g.part + (int64_t)blockIdx.x * (TI * TJ * 64 * NW) + tid;   // [split][tile]
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) to[(i * TJ + j) * 64 * NW] = acc[i][j];
    return;
  }
  block_sync();   // the last operands have been read
  epilogue<MODE, TI, TJ>(g, acc, in, (char *)s_t + wave * (TI * TJ * 512), n0 + wn * TI * 16,
                         m0 + wm * TJ * 16);
}

// The tiles' sums from their splits, exact in any order, and the epilogue.
template <int MODE, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void int8_join_kernel(I8Args g) {
  constexpr int NW = WN * WM, TI = BN / WN / 16, TJ = BM / WM / 16;
  __shared__ __align__(1024) uint4 s_t[NW * TI * TJ * 32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t n0, m0;
  tile_of<BN, BM>(g, blockIdx.x, n0, m0);
  n0 += (wave % WN) * TI * 16;
  m0 += (wave / WN) * TJ * 16;
  EpilogueIn<MODE, TI, TJ> in;
  in.load(g, n0, m0);
  i32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const i32x4 *from = g.part + (int64_t)blockIdx.x * (TI * TJ * 64 * NW) + threadIdx.x;
#pragma unroll 2
  for (int y = 0; y < g.S; ++y, from += (int64_t)gridDim.x * (TI * TJ * 64 * NW))
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] += from[(i * TJ + j) * 64 * NW];
  epilogue<MODE, TI, TJ>(g, acc, in, (char *)s_t + wave * (TI * TJ * 512), n0, m0);
}

// ---- decode: up to 16 tokens ------------------------------------------------
// A workgroup of eight waves owns 16 NR rows of the weight and all tokens; the
// waves take 128-code steps in turn and their int32 sums meet in LDS. Bound by
// the weight's bytes, each read once: a wave fetches its steps by LDS DMA, 8 rows
// x 128 bytes at a time (whole lines; the 16 rows x 64 bytes of an operand read
// as half lines take a third longer), ST steps ahead in slots of its own, so
// that no barrier is needed. The tokens' codes come from L2 as often as there
// are workgroups. Wave w also takes ranks 16 w .. +15 of the rank-r term, whose
// operands it loads up front.
struct I8Gemv {
  const int8_t *W;
  const float *sw;
  int64_t d, k;
  const int8_t *In;      // M x ldi
  int64_t ldi;
  const float *sx;
  int M;
  const uint16_t *B;     // d x r
  const uint16_t *hi, *lo;   // M x rp: s H
  int r, rp;
  uint16_t *Y;           // M x d
};

constexpr int GV_W = 8;

template <int NR, int ST>
__global__ __launch_bounds__(64 * GV_W) void int8_gemv_kernel(I8Gemv g) {
  constexpr int SLOT = NR * 16 * BK;           // bytes of a step's rows
  constexpr int RED = GV_W * NR * 256 * 8;     // sums: int32, and float32 of the ranks
  constexpr int LDS = GV_W * ST * SLOT > RED ? GV_W * ST * SLOT : RED;
  __shared__ __align__(1024) char s_t[LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, grp = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NR;
  const int m = c16 < g.M ? c16 : g.M - 1;
  const int8_t *const x = g.In + m * g.ldi + 16 * grp;
  int64_t row[NR];
#pragma unroll
  for (int b = 0; b < NR; ++b) row[b] = n0 + 16 * b + c16 < g.d ? n0 + 16 * b + c16 : g.d - 1;
  // DMA sources: rows 8 i .. +7 of the block, whose chunks are permuted as in
  // the GEMM's tiles; past the matrix the last valid piece, against zero codes
  const int8_t *w[2 * NR];
  uint32_t wc[2 * NR];
#pragma unroll
  for (int i = 0; i < 2 * NR; ++i) {
    const int r = 8 * i + (lane >> 3);
    w[i] = g.W + (n0 + r < g.d ? n0 + r : g.d - 1) * g.k;
    wc[i] = 16 * swz(r & 15, lane & 7);
  }
  const int nk = (int)ql_cdiv(g.k, BK), mine = nk > wave ? (nk - wave + GV_W - 1) / GV_W : 0;
  const uint32_t slots = lds_addr(s_t) + wave * ST * SLOT, end = (uint32_t)g.k - 16;
  auto issue = [&](int step) {   // this wave's step-th
    const uint32_t kk = (uint32_t)(wave + step * GV_W) * BK;
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i) {
      const uint32_t at = kk + wc[i] < end ? kk + wc[i] : end;
      dma16(w[i] + at, __builtin_amdgcn_readfirstlane(slots + (step % ST) * SLOT + 1024 * i));
    }
  };
  // ranks 16 wave .. +15: lanes 0-31 against the high parts, 32-63 the low
  const bool lr = 16 * wave < g.rp;
  uint4 lv[NR], sv = ql::zero4();
  if (lr) {
    const int t = 16 * wave + 8 * (grp & 1);
    sv = *(const uint4 *)((grp < 2 ? g.hi : g.lo) + (int64_t)m * g.rp + t);
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      if (g.r % 8 == 0) {
        lv[b] = t < g.r ? *(const uint4 *)(g.B + row[b] * g.r + t) : ql::zero4();
      } else {
        uint32_t e[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int tc = t + y < g.r ? t + y : g.r - 1;
          e[y] = g.B[row[b] * g.r + tc];
          e[y] = t + y < g.r ? e[y] : 0u;
        }
        lv[b] = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16),
                           e[6] | (e[7] << 16));
      }
    }
  }
  // the tokens' codes of a step, beside its DMAs
  i32x4 xv[ST][SL];
  auto tokens = [&](int buf, int step) {
    const int kk = (wave + step * GV_W) * BK;
#pragma unroll
    for (int c = 0; c < SL; ++c) xv[buf][c] = *(const i32x4 *)(x + kk + 64 * c);
  };
  i32x4 acc[NR];
#pragma unroll
  for (int b = 0; b < NR; ++b) acc[b] = i32x4{0, 0, 0, 0};
  // A step's DMAs and token loads go out ST steps ahead; they retire in order.
  constexpr int OPS = 2 * NR + SL;
#pragma unroll
  for (int u = 0; u < ST; ++u)
    if (u < mine) {
      issue(u);
      tokens(u, u);
    }
  for (int s0 = 0; s0 < mine; s0 += ST) {
#pragma unroll
    for (int u = 0; u < ST; ++u) {
      if (s0 + u >= mine) break;
      if (s0 + u + ST - 1 < mine) wait_vm_le<(ST - 1) * OPS>();
      else wait_vm_le<0>();
      asm volatile("" ::: "memory");
      const char *ws = s_t + wave * ST * SLOT + u * SLOT;
#pragma unroll
      for (int c = 0; c < SL; ++c)
#pragma unroll
        for (int b = 0; b < NR; ++b)
          acc[b] = mfma_i8(*(const i32x4 *)(ws + (16 * b + c16) * BK + 16 * swz(c16, 4 * c + grp)),
                           xv[u][c], acc[b]);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);   // the slot has been read
      if (s0 + u + ST < mine) {
        issue(s0 + u + ST);
        tokens(u, s0 + u + ST);
      }
    }
  }
  block_sync();   // by every wave: the sums take their place
  int(*const s_red)[NR][4][64] = (int(*)[NR][4][64])s_t;
  float(*const s_lr)[NR][4][64] = (float(*)[NR][4][64])(s_t + GV_W * NR * 1024);
#pragma unroll
  for (int b = 0; b < NR; ++b) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s_red[wave][b][q][lane] = acc[b][q];
    if (lr) {
      const f32x4 t = ql::mfma16(lv[b], sv, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
      for (int q = 0; q < 4; ++q) s_lr[wave][b][q][lane] = t[q];
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * NR; o += 64 * GV_W) {
    const int n = o % (16 * NR), t = o / (16 * NR), b = n >> 4;
    if (t >= g.M || n0 + n >= g.d) continue;
    const int q = n & 3, l = 16 * ((n & 15) >> 2) + t;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < GV_W; ++v) sum += s_red[v][b][q][l];
    const float2 s = token_scale(g.sx[t]);
    float y = (float)sum * s.x * g.sw[n0 + n] * s.y;
    for (int v = 0; 16 * v < g.rp; ++v) y += s_lr[v][b][q][l];
    g.Y[(int64_t)t * g.d + n0 + n] = ql::f_to_bf16(y);
  }
}

// ---- host -----------------------------------------------------------------------
// Tile and splits of a product of M tokens, N columns, K codes, by the least
// time of what was measured, in us: a workgroup takes a fixed time for its start
// and end and a time per K-step that grows by a quarter as the chip fills; a
// split adds the partial sums' way through memory and the join. Measured, the
// tiles 128 x 256 / 128 x 128 / the chosen one with its join: 4096 x 4096, 64
// tokens 27 / 17 / 11.0 (128 x 64, three splits; four, by the model a hundredth
// slower, 10.6), 128 tokens 27 / 17 / 13.2 (128 x 64), 512 28 / 18, 2048 35 / 39;
// 4096 x 11008, 128 tokens 63 / 37 / 18.3 (128 x 64, four splits), 256 64 / 38 / 23
// (128 x 128, four splits), 777 69 / 45; 11008 x 4096, 2048 tokens 92 / 109.
struct I8Plan {
  int cfg;        // 0: 128 x 256, 1: 128 x 128, 2: 128 x 64 (columns x tokens)
  int S;
  int64_t tiles, part;   // part: bytes of partial sums
};
I8Plan i8_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t tn = ql_cdiv(N, 128), nk = ql_cdiv(K, BK);
  constexpr double kFixed[3] = {7.3, 5.2, 4.2}, kStep[3] = {0.65, 0.365, 0.268};
  I8Plan best{0, 1, tn * ql_cdiv(M, 256), 0};
  double least = -1.0;
  for (int cfg = 0; cfg < 3; ++cfg) {
    const int64_t bm = cfg == 0 ? 256 : cfg == 1 ? 128 : 64, tiles = tn * ql_cdiv(M, bm);
    if (cfg == 2 && M > 128) continue;
    for (int S : {1, 2, 3, 4, 6, 8}) {
      if (S > 1 && (cfg == 0 || S * 2 > nk)) break;
      if (tiles * S >= int64_t(1) << 23) break;   // 2^32 threads; 128 x 256 tiles stay below
      const int64_t wgs = tiles * S, bytes = wgs * bm * 128 * 4;
      const double fill = wgs < 256 ? (double)wgs / 256.0 : 1.0;
      double t = (double)ql_cdiv(wgs, 256) *
                 (kFixed[cfg] + kStep[cfg] * (1.0 + 0.26 * fill) * (double)ql_cdiv(nk, S));
      if (S > 1) t += 1.0 + (double)bytes / (cfg == 2 ? 1.25e6 : 1.85e6);
      if (least < 0.0 || t < least) {
        least = t;
        best = I8Plan{cfg, S, tiles, S > 1 ? bytes : 0};
      }
    }
  }
  return best;
}

template <int MODE, int BM, int WN, int WM, int NST>
void launch_cfg(const I8Args &g, const I8Plan &p, hipStream_t st) {
  constexpr int NTH = 64 * WN * WM;
  if (p.S == 1) {
    int8_gemm_kernel<MODE, 128, BM, WN, WM, NST, false><<<(unsigned)p.tiles, NTH, 0, st>>>(g);
  } else {
    int8_gemm_kernel<MODE, 128, BM, WN, WM, NST, true>
        <<<(unsigned)(p.tiles * p.S), NTH, 0, st>>>(g);
    int8_join_kernel<MODE, 128, BM, WN, WM><<<(unsigned)p.tiles, NTH, 0, st>>>(g);
  }
}

template <int MODE>
void launch_mode(const I8Args &g, const I8Plan &p, hipStream_t st) {
  if (p.cfg == 0)
    int8_gemm_kernel<MODE, 128, 256, 4, 2, 3, false><<<(unsigned)p.tiles, 512, 0, st>>>(g);
  else if (p.cfg == 1) launch_cfg<MODE, 128, 4, 2, 4>(g, p, st);
  else launch_cfg<MODE, 64, 4, 2, 6>(g, p, st);
}

}  // namespace

size_t int8_gemm_part_bytes(int64_t M, int64_t N, int64_t K) {
  return (size_t)i8_plan(M, N, K).part;
}

// The partial sums grow and fall with M. A plan is the same for 1 to 64 tokens,
// 65 to 128, and every 128 from there. By the times above a split saves at most
// the idle part of a round, kFixed + 0.46 nk us, and adds at least
// tiles (kFixed / 256 + 0.07) us, so that none is taken past 256 + 6 nk tiles.
size_t int8_gemm_part_bytes_upto(int64_t M, int64_t N, int64_t K) {
  const int64_t tn = ql_cdiv(N, 128), most = 256 + 6 * ql_cdiv(K, BK);
  int64_t bytes = 0;
  for (int64_t m = 1; m <= M && tn * (m / 128) <= most; m = m == 1 ? 65 : m == 65 ? 129 : m + 128) {
    const int64_t part = i8_plan(m, N, K).part;
    bytes = part > bytes ? part : bytes;
  }
  return (size_t)bytes;
}

qlora_status launch_int8_gemm(int mode, const int8_t *W, const float *sw, int64_t d, int64_t k,
                              const int8_t *In, int64_t ldi, const float *sx, int64_t M,
                              const uint16_t *L, int ldl, const uint16_t *hi, const uint16_t *lo,
                              int rp, uint16_t *Out, void *part, hipStream_t st) {
  const int64_t N = mode == 0 ? d : k, K = mode == 0 ? k : d;
  const I8Plan p = i8_plan(M, N, K);
  const I8Args g{W, sw, d, k, In, ldi, sx, M, N, K, L, ldl, hi, lo, rp, Out, p.S, (i32x4 *)part};
  QlProf prof(mode == 0 ? QLORA_K_INT8_GEMM_FWD : QLORA_K_INT8_GEMM_DX, st);
  if (mode == 0) launch_mode<0>(g, p, st);
  else launch_mode<1>(g, p, st);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}

qlora_status launch_int8_gemv(const int8_t *W, const float *sw, int64_t d, int64_t k,
                              const int8_t *In, int64_t ldi, const float *sx, int64_t M,
                              const uint16_t *B, const uint16_t *hi, const uint16_t *lo, int r,
                              int rp, uint16_t *Y, hipStream_t st) {
  const I8Gemv g{W, sw, d, k, In, ldi, sx, (int)M, B, hi, lo, r, rp, Y};
  QlProf prof(QLORA_K_INT8_GEMV, st);
  // two row blocks a workgroup once one fills the chip twice
  if (d >= 8192) int8_gemv_kernel<2, 2><<<(unsigned)ql_cdiv(d, 32), 64 * GV_W, 0, st>>>(g);
  else int8_gemv_kernel<1, 4><<<(unsigned)ql_cdiv(d, 16), 64 * GV_W, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}
