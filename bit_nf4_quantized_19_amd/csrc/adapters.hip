// Plan of a batch whose tokens use different adapters, gfx950.
//
// A stable counting sort of the tokens by adapter, in one workgroup: the
// kernels that follow (lora_small.hip, gemm.hip) then work on runs of one
// adapter's tokens whatever order the batch has, and sum each adapter's
// gradient over its tokens in batch order. The lists they index by workgroup
// (groups of AD_TOK tokens, splits of an adapter's tokens) are written in the
// same pass: position p of an adapter whose first position is off opens group
// (p - off) / AD_TOK when that division is exact, and likewise its splits.
// Group g of G has record (g % (G / 8)) 8 + g / (G / 8): workgroups go to the
// eight XCDs in turn, so the groups of one adapter, which are neighbours, meet
// in one XCD's L2.
//
// Each of the 8 waves owns one contiguous eighth of the batch and one row of
// an LDS histogram (8 x 1025 counters is the most that leaves room for the
// per-adapter tables in 64 KB). A step takes 64 tokens: the lanes of one
// adapter find each other by ballots over the bits of its number, and the
// first of them moves the counter, so a counter is touched once per step and
// adapter and every token's place is fixed by its index. The batch is read
// twice (count, place); the time is the latency of that chain, not bytes, and
// a batch pays it once for all its linears.
#include "../../include/qlora_adapters.h"
#include "kernels.h"

namespace {

constexpr int PT = 512, PW = PT / 64;
constexpr int PB = QLORA_MAX_ADAPTERS + 1;   // buckets: adapters, then none

struct PlanArgs {
  const int32_t *ids;
  int64_t M, split_tok, max_groups;
  int n;
  int *tok, *perm, *sid, *off, *num, *grp, *split;
};

// Lanes of the wave that hold the same bucket (bits of it that can be set).
QL_DEV uint64_t same_bucket(int b, int bits) {
  uint64_t m = ~0ull;
  for (int i = 0; i < bits; ++i) {
    const uint64_t v = __ballot((b >> i) & 1);
    m &= ((b >> i) & 1) ? v : ~v;
  }
  return m;
}

// Exclusive sum over the workgroup's threads; `total` receives the whole sum.
QL_DEV int block_exsum(int v, int *tmp, int tid, int &total) {
  const int lane = tid & 63, wave = tid >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();   // tmp may still be read from the previous call
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  int base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < PW; ++w) {
    if (w < wave) base += tmp[w];
    total += tmp[w];
  }
  return base + x - v;
}

__global__ __launch_bounds__(PT) void adapter_plan_kernel(PlanArgs g) {
  __shared__ int hist[PW][PB];                       // counts, then next positions
  __shared__ int s_off[PB + 1], s_grp[PB], s_split[PB], s_slot[PB];
  __shared__ int s_per;                              // groups of one eighth of the records
  __shared__ int tmp[PW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = g.n, nb = n + 1;
  for (int i = tid; i < PW * PB; i += PT) hist[i / PB][i % PB] = 0;
  __syncthreads();

  const int64_t per = ql_rup(ql_cdiv(g.M, PW), 64);
  const int64_t lo = wave * per, hi = min(g.M, lo + per);
  const uint64_t below = (1ull << lane) - 1;
  // bucket of token m; lanes past the end join no one (bucket nb is never counted)
  auto bucket = [&](int64_t m) -> int {
    if (m >= hi) return nb;
    const int id = g.ids[m];
    return (id >= 0 && id < n) ? id : n;
  };
  const int mbits = 32 - __builtin_clz(nb);
  for (int64_t m0 = lo; m0 < hi; m0 += 64) {
    const int b = bucket(m0 + lane);
    const uint64_t same = same_bucket(b, mbits);
    if (b < nb) {
      if ((same & below) == 0) atomicAdd(&hist[wave][b], __popcll(same));
      g.tok[m0 + lane] = b < n ? b : -1;
    }
  }
  __syncthreads();

  // per bucket: first position, groups, splits and slots before it
  constexpr int PER = (PB + PT - 1) / PT;
  int cnt[PER], c4[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    int c = 0;
    if (b < nb)
      for (int w = 0; w < PW; ++w) c += hist[w][b];
    cnt[i] = c;
    const int ns = b < n ? max(1, (int)ql_cdiv(c, g.split_tok)) : 0;
    c4[0] += c;
    c4[1] += (int)ql_cdiv(c, AD_TOK);
    c4[2] += ns;
    c4[3] += ns > 1 ? ns : 0;
  }
  int tot[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) c4[q] = block_exsum(c4[q], tmp, tid, tot[q]);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b >= nb) break;
    const int c = cnt[i], ns = b < n ? max(1, (int)ql_cdiv(c, g.split_tok)) : 0;
    s_off[b] = g.off[b] = c4[0];
    s_grp[b] = c4[1];
    s_split[b] = c4[2];
    s_slot[b] = ns > 1 ? c4[3] : -1;
    if (b < n && c == 0) {   // an empty adapter's split: its gradients are written as zeros
      int *e = g.split + 8 * (int64_t)c4[2];
      e[0] = b; e[1] = c4[0]; e[2] = c4[0]; e[3] = -1; e[4] = 0; e[5] = 1; e[6] = 0; e[7] = 0;
    }
    int p = c4[0];
    for (int w = 0; w < PW; ++w) {   // the waves' tokens follow each other
      const int x = hist[w][b];
      hist[w][b] = p;
      p += x;
    }
    c4[0] += c;
    c4[1] += (int)ql_cdiv(c, AD_TOK);
    c4[2] += ns;
    c4[3] += ns > 1 ? ns : 0;
  }
  if (tid == 0) {
    s_off[nb] = g.off[nb] = (int)g.M;
    g.num[0] = tot[2];
    g.num[1] = g.num[2] = g.num[3] = 0;
    s_per = (int)ql_cdiv(tot[1], 8);
  }
  // records without a group (group (i % 8) per + i / 8 would be past the last)
  const int per8 = (int)ql_cdiv(tot[1], 8);
  for (int64_t i = tid; i < g.max_groups; i += PT)
    if (i >= 8 * (int64_t)per8 || (i & 7) * (int64_t)per8 + (i >> 3) >= tot[1])
      g.grp[AD_GRP * i + 2] = 0;
  __syncthreads();

  for (int64_t m0 = lo; m0 < hi; m0 += 64) {
    const int b = bucket(m0 + lane);
    const uint64_t same = same_bucket(b, mbits);
    const int first = __builtin_ctzll(same);
    int base = 0;
    if (b < nb && lane == first) base = atomicAdd(&hist[wave][b], __popcll(same));
    base = __shfl(base, first);
    if (b >= nb) continue;
    const int p = base + __popcll(same & below);
    g.perm[p] = (int)(m0 + lane);
    g.sid[p] = b < n ? b : -1;
    const int q = p - s_off[b], end = s_off[b + 1];
    const int gi = s_grp[b] + q / AD_TOK;
    int *e = g.grp + AD_GRP * ((int64_t)(gi % s_per) * 8 + gi / s_per);
    e[4 + q % AD_TOK] = (int)(m0 + lane);
    if (q % AD_TOK == 0) {
      e[0] = b;
      e[1] = p;
      e[2] = min(AD_TOK, end - p);
    }
    if (b < n && q % (int)g.split_tok == 0) {
      const int i = q / (int)g.split_tok;
      int *e = g.split + 8 * (int64_t)(s_split[b] + i);
      e[0] = b;
      e[1] = p;
      e[2] = (int)min<int64_t>(p + g.split_tok, end);
      e[3] = s_slot[b];
      e[4] = i;
      e[5] = (int)ql_cdiv(end - s_off[b], g.split_tok);
      e[6] = 0;
      e[7] = 0;
    }
  }
}

}  // namespace

// split_tok: an adapter that holds the whole batch is cut into AD_SPLITS
// ranges (the token splits the single-adapter gradient uses at 4096 x 4096),
// never finer than its smallest chunk.
AdapterPlan::AdapterPlan(void *data, int64_t M_, int n_) : M(M_), n(n_) {
  split_tok = ql_rup(ql_cdiv(M, AD_SPLITS), 128);
  max_groups = ql_rup(M / AD_TOK + (M < n + 1 ? M : n + 1), 8);
  max_splits = M / split_tok + n;
  max_slots = 2 * ql_cdiv(M, split_tok);
  int64_t at = 0;
  auto take = [&](int64_t ints) {
    int *p = data ? (int *)data + at : nullptr;
    at += ql_rup(ints, 64);
    return p;
  };
  tok = take(M);
  perm = take(M);
  sid = take(M);
  off = take(n + 2);
  num = take(4);
  grp = take(AD_GRP * max_groups);
  split = take(8 * max_splits);
  bytes = (size_t)at * 4;
}

qlora_status launch_adapter_plan(const int32_t *ids, const AdapterPlan &p, hipStream_t st) {
  PlanArgs g{ids, p.M, p.split_tok, p.max_groups, p.n, p.tok, p.perm, p.sid, p.off, p.num, p.grp, p.split};
  QlProf prof(QLORA_K_ADAPTER_PLAN, st);
  adapter_plan_kernel<<<1, PT, 0, st>>>(g);
  QL_LAUNCH_CHECK();
  return QLORA_OK;
}
