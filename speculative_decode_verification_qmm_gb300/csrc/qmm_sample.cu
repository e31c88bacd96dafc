// qmm_sample.cu -- verification of a drafted tree by rejection sampling
// (qmm_verify_sample in include/qmm.h).
//
// Mathematics.  With P and Q the target's and the drafter's softmax at the
// current node, a child with token x is accepted with probability min(1, P(x) /
// Q(x)); a rejected one leaves P' = max(P - Q, 0) / Z and Q' = Q without x / ZQ,
// so the next sibling, which was drawn from Q', is tried against P', and the
// token emitted where the walk ends is a draw from the target.  That draw is an
// exponential race, argmax P(v) / noise(v): unlike an inverted cumulative sum
// it does not depend on the order of a sum over the vocabulary.
//
// A softmax value needs its row's maximum and sum; a sibling after a rejection
// needs Z and ZQ.  Everything else about a decision is scalar.  P and Q after r
// rejections are recomputed per entry from the scores and the r pairs (Z, ZQ),
// so no vocabulary-sized state is kept and a row is read from HBM once and
// from L2 afterwards.  A cluster of CTAs walks one sequence: each CTA takes a
// share of the vocabulary, and sums cross the cluster through distributed
// shared memory, one cluster barrier each.
//
// Only rows of visited nodes matter, but they are known one after the other.
// With few bytes in the batch's rows a first kernel takes the statistics of
// every row that could be visited, over the whole GPU, and the walk needs no
// pass until its end (EAGER); with many, the walk reads the rows of its own
// nodes only, four nodes ahead along the first children.  sample_eager() holds
// the rule.
// What bounds it: a chain of dependent steps.  Measured, target and drafter
// scores of 151,936 entries: one sequence, chain of 8, fp32: 10.3 us, two launches
// of which the first reads 8.5 MB; 32 sequences, chains of 16, 16 bits: 69 us, the
// steps of the longest walks, where the visited rows of all sequences take 14 at
// the copy rate: the busiest SMs issue in 93 % of their cycles, all of them in 30 %
// on average; 4 trees of 64, 50,257 fp32: 13.1 us.
// 16-byte copies where rows lie on 16-byte boundaries (WIDE), else single entries
// in the passes over whole rows of a walk: 70 us against 81 for the batch above.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {
namespace {

constexpr int MAX_T = QMM_TREE_MAX_T;
constexpr int STAT_THREADS = 256;
constexpr int STAT_DEPTH = 8;  // steps of a thread's ring
constexpr int WALK_THREADS = 512;
constexpr int WALK_DEPTH = 8;  // 16-byte slots of a thread's ring: 64 KB a CTA, two CTAs on an SM (12: 73 us for 69)
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_CHUNKS = 32;  // parts of a row in the eager statistics
constexpr int AHEAD = 4;        // nodes whose rows the walk reads at a time

struct SampleParams {
  const void* target;
  const void* draft;
  int64_t t_sb, t_st, d_sb, d_st;
  int64_t V;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* n_tokens;
  const float* u;
  const float* noise;
  const float* temperature;
  int32_t* accept;
  int32_t* path;
  float2* stats;  // eager: [B][T][target, draft][chunks] (maximum, sum)
  int T;
  int chunks;
};

template <int DT>
struct Score;
template <>
struct Score<QMM_DT_F32> {
  using type = float;
  static constexpr int VEC = 4;
};
template <>
struct Score<QMM_DT_BF16> {
  using type = uint16_t;
  static constexpr int VEC = 8;
};
template <>
struct Score<QMM_DT_F16> {
  using type = uint16_t;
  static constexpr int VEC = 8;
};

template <int DT>
__device__ __forceinline__ float score_at(const void* row, int64_t v) {
  if constexpr (DT == QMM_DT_F32)
    return __ldg(static_cast<const float*>(row) + v);
  else
    return unpack16<DT == QMM_DT_BF16>(__ldg(static_cast<const uint16_t*>(row) + v));
}

// N consecutive scores from a ring's slot of 16 bytes.
template <int DT, int N>
__device__ __forceinline__ void ring_scores(uint32_t slot, float (&x)[N]) {
  const uint4 a = lds128(slot);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == QMM_DT_F32) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = unpack16<DT == QMM_DT_BF16>((uint16_t)(w[i] & 0xFFFFu));
      x[2 * i + 1] = unpack16<DT == QMM_DT_BF16>((uint16_t)(w[i] >> 16));
    }
  }
}

// Running (base, sum of 2^(x c - base)) over a share of a row's scores x, with c =
// log2(e) / temperature > 0 and base = max(x) c, rounded.  x c - base is one FMA;
// because sums, probabilities and joins all use the rounded bases, that rounding
// cancels between them.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  // a part whose base is -inf has no mass (its sum is 0, or NaN for NaN scores)
  r.s = (a.m == -INFINITY ? a.s : a.s * ex2(a.m - r.m)) + (b.m == -INFINITY ? b.s : b.s * ex2(b.m - r.m));
  return r;
}

// Thread-private rings in shared memory: each thread copies what it will read, a
// few steps ahead (cp.async), so that a step waits for nothing but its own copy
// and no barrier is needed.  A thread's slots lie THREADS * 16 bytes apart.
template <int THREADS, int SLOTS>
struct Ring {
  uint32_t base, at;
  __device__ __forceinline__ explicit Ring(uint32_t smem) : base(smem + threadIdx.x * 16), at(base) {}
  template <int BY>
  __device__ __forceinline__ void next() {
    at += BY * THREADS * 16;
    if (at == base + SLOTS * THREADS * 16) at = base;
  }
};

// The statistics of a thread's share of a row: granules (16 bytes, counted from
// the one that holds the row's first entry, so that any alignment will do) g,
// g + stride, ... < end, four at a time: the maximum and the exponentials of 32
// (16) entries overlap, where one granule at a time left the SM waiting for
// chains of dependent instructions.
template <int DT, int THREADS, int SLOTS>
__device__ __forceinline__ MaxSum row_share(uint32_t smem, const void* row, int V, int g, int end, int stride,
                                            float c) {
  constexpr int SIZE = (int)sizeof(typename Score<DT>::type), N = 16 / SIZE, U = 4;
  constexpr uint32_t SLOT = THREADS * 16;
  static_assert(SLOTS % U == 0, "whole steps");
  const int skip = (int)((uintptr_t)row & 15);
  const int last = (int)((skip + (int64_t)V * SIZE + 15) / 16);
  end = end < last ? end : last;
  const char* from = reinterpret_cast<const char*>(row) - skip + (int64_t)g * 16;
  const int64_t hop = (int64_t)stride * 16;
  Ring<THREADS, SLOTS> in(smem), out(smem);
  int ig = g;
  auto issue = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ig < end) cp_async16(in.at + u * SLOT, from, 16);
      ig += stride;
      from += hop;
    }
    cp_async_commit();
    in.template next<U>();
  };
#pragma unroll
  for (int i = 0; i < SLOTS / U - 1; ++i) issue();
  MaxSum a{-INFINITY, 0.f};
  for (; g < end; g += U * stride) {
    issue();
    cp_async_wait<SLOTS / U - 1>();
    float x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gu = g + u * stride;
      if (gu < end) {
        ring_scores<DT, N>(out.at + u * SLOT, x[u]);
        if (gu == 0 || gu + 1 == last) {
          const int v = gu * N - skip / SIZE;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (v + e < 0 || v + e >= V) x[u][e] = -INFINITY;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[u][e] = -INFINITY;
      }
    }
    out.template next<U>();
    float mx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mx[u] = x[u][0];
#pragma unroll
      for (int e = 1; e < N; ++e) mx[u] = fmaxf(mx[u], x[u][e]);
    }
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
    if (top > a.m) {
      a.s = a.m == -INFINITY ? a.s : a.s * ex2(a.m - top);
      a.m = top;
    }
    const float base = a.m == -INFINITY ? 0.f : a.m;
    const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
    float2 sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u] = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float2 y = fma2(make_float2(x[u][e], x[u][e + 1]), c2, b2);
        y.x = ex2(y.x);
        y.y = ex2(y.y);
        sum[u] = __fadd2_rn(sum[u], y);
      }
    }
    const float2 y = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
    a.s += y.x + y.y;
  }
  cp_async_wait<0>();
  return a;
}

// Granules of 16 bytes that a row of any alignment spans at most.
__host__ __device__ constexpr int row_granules(int64_t V, int size) { return (int)((V * size + 15) / 16 + 1); }

__device__ __forceinline__ MaxSum warp_join(MaxSum a) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    MaxSum o;
    o.m = __shfl_xor_sync(0xFFFFFFFFu, a.m, d);
    o.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, d);
    a = join(a, o);
  }
  return a;
}

__device__ __forceinline__ void prefetch_l2(const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); }

__device__ __forceinline__ float log2e_over(const float* temperature, int b) {
  return 1.4426950408889634f / (temperature ? __ldg(temperature + b) : 1.f);
}

// ---------------------------------------------------------------- statistics
// CTA (chunk, row, sequence): (maximum, sum) of one part of row node = y / 2 of
// target (y even) or draft, if the node has children.
template <int DT>
__global__ void __launch_bounds__(STAT_THREADS) sample_stats_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  using E = typename Score<DT>::type;
  __shared__ MaxSum s_part[STAT_THREADS / 32];
  const int b = blockIdx.z, tid = threadIdx.x;
  const int sides = p.draft ? 2 : 1;
  const int node = blockIdx.y / sides, side = blockIdx.y % sides;
  const int n = p.n_tokens ? min(__ldg(p.n_tokens + b), p.T) : p.T;
  bool child = false;
  if (p.parents)
    child = tid > node && tid < n && __ldg(p.parents + (int64_t)b * p.T + tid) == node;
  else
    child = node + 1 < n;
  pdl_trigger();
  if (!__syncthreads_or(child)) return;
  const E* row = side ? static_cast<const E*>(p.draft) + b * p.d_sb + node * p.d_st
                      : static_cast<const E*>(p.target) + b * p.t_sb + node * p.t_st;
  const float c = log2e_over(p.temperature, b);
  const int64_t groups = row_granules(p.V, (int)sizeof(E));
  const int g0 = (int)(groups * blockIdx.x / p.chunks), g1 = (int)(groups * (blockIdx.x + 1) / p.chunks);
  MaxSum a = row_share<DT, STAT_THREADS, STAT_DEPTH>(smem_u32(ring), row, (int)p.V, g0 + tid, g1, STAT_THREADS, c);
  a = warp_join(a);
  if ((tid & 31) == 0) s_part[tid >> 5] = a;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < STAT_THREADS / 32; ++w) a = join(a, s_part[w]);
    p.stats[(((int64_t)b * p.T + node) * 2 + side) * p.chunks + blockIdx.x] = make_float2(a.m, a.s);
  }
}

// ---------------------------------------------------------------- the walk
struct WalkSmem {
  float tx[MAX_T], qx[MAX_T];        // scores of node i's token at its parent
  float u[MAX_T];
  int token[MAX_T], parent[MAX_T], path[MAX_T];
  float pm[MAX_T], ps[MAX_T], qm[MAX_T], qs[MAX_T];  // eager: row maxima and 1 / sums
  float rz[MAX_T], rzq[MAX_T];       // rejections at the current node: 1 / Z (0: P kept), 1 / ZQ
  int rx[MAX_T];                     // and their tokens
  int list[AHEAD];                   // nodes whose rows are read together
  float2 part[2 * AHEAD][WALK_THREADS / 32];  // per warp
  float4 cl[2][AHEAD];               // this CTA's part of cluster sums, two in turn
};

template <int DT, bool WIDE, bool EAGER>
__global__ void __launch_bounds__(WALK_THREADS, 2) sample_walk_kernel(const __grid_constant__ SampleParams p,
                                                                      int cluster) {
  constexpr int N = WIDE ? Score<DT>::VEC : 1;
  using E = typename Score<DT>::type;
  __shared__ WalkSmem s;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  const uint32_t ring = smem_u32(ring_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / cluster;
  const int rank = blockIdx.x - b * cluster;
  const int T = p.T;
  int n = p.n_tokens ? __ldg(p.n_tokens + b) : T;
  n = n < 0 ? 0 : (n > T ? T : n);
  const float c = log2e_over(p.temperature, b);
  const bool has_q = p.draft != nullptr;
  const E* target = static_cast<const E*>(p.target) + b * p.t_sb;
  const E* draft = has_q ? static_cast<const E*>(p.draft) + b * p.d_sb : nullptr;
  const float* noise = p.noise + (int64_t)b * p.V;

  for (int i = tid; i < MAX_T; i += WALK_THREADS) {
    s.parent[i] = -1;
    if (i >= T) continue;
    const int par = p.parents ? __ldg(p.parents + (int64_t)b * T + i) : i - 1;
    const int x = __ldg(p.tokens + (int64_t)b * T + i);
    const bool valid = i > 0 && i < n && par >= 0 && par < i && x >= 0 && x < p.V;
    s.parent[i] = valid ? par : -1;
    s.token[i] = x;
    s.u[i] = __ldg(p.u + (int64_t)b * T + i);
    s.tx[i] = valid ? score_at<DT>(target + par * p.t_st, x) : 0.f;
    s.qx[i] = valid && has_q ? score_at<DT>(draft + par * p.d_st, x) : 0.f;
    s.path[i] = -1;
  }
  if constexpr (EAGER) {
    pdl_wait();  // the statistics of the first kernel
    for (int r = warp; r < 2 * T; r += WALK_THREADS / 32) {
      const int node = r >> 1, side = r & 1;
      if (side && !has_q) continue;
      MaxSum a{-INFINITY, 0.f};
      if (lane < p.chunks) {
        const float2 v = __ldcg(p.stats + (((int64_t)b * T + node) * 2 + side) * p.chunks + lane);
        a.m = v.x, a.s = v.y;
      }
      a = warp_join(a);
      if (lane == 0) {
        (side ? s.qm : s.pm)[node] = a.m == -INFINITY ? 0.f : a.m;
        (side ? s.qs : s.ps)[node] = a.s != 0.f ? 1.f / a.s : 0.f;
      }
    }
  }
  __syncthreads();

  // Reductions over the cluster.  Every warp leaves a value in s.part[i]; warp i
  // adds up the CTA's, then, after a barrier of the cluster, the ranks', each
  // with `op` over the lanes in an order that the sizes fix.  The buffers
  // alternate, so that one barrier a reduction is enough.  These barriers have no
  // limit: every thread of the cluster meets them in the same order because each
  // decides alike, from values in its own CTA's memory that were computed from
  // the same inputs in the same order and are not written while any warp reads them.
  int turn = 0;
  constexpr int WARPS = WALK_THREADS / 32;
  auto reduce = [&](int count, auto none, auto op) {
    using X = decltype(none);  // float2, or float4 where count is at most AHEAD
    X* part = reinterpret_cast<X*>(s.part);
    X* sums = reinterpret_cast<X*>(s.cl[turn]);
    __syncthreads();
    X x = none;
    if (warp < count) {
      if (lane < WARPS) x = part[warp * WARPS + lane];
      x = op(x);
      if (lane == 0) sums[warp] = x;
    }
    cluster_sync_all();
    x = none;
    if (warp < count) {
      if (lane < cluster) {
        const uint32_t a = dsmem_map(smem_u32(sums + warp), lane);
        x.x = ld_dsmem_f32(a);
        x.y = ld_dsmem_f32(a + 4);
        if constexpr (sizeof(X) > 8) x.z = ld_dsmem_f32(a + 8);
      }
      x = op(x);
    }
    turn ^= 1;
    return x;  // of reduction `warp`, in its lanes
  };
  static_assert(2 * AHEAD <= WARPS, "a warp for each value");

  const int v0 = (rank * WALK_THREADS + tid) * N, step = cluster * WALK_THREADS * N, vend = (int)p.V;

  // The whole noise row is read in the end.
  for (int v = (rank * WALK_THREADS + tid) * 32; v < vend; v += cluster * WALK_THREADS * 32)
    prefetch_l2(noise + v);

  int node = 0, k = 0, rej = 0;
  float pm = 0.f, ps = 0.f, qm = 0.f, qs = 0.f;
  uint64_t known = EAGER ? ~0ull : 0ull;  // nodes whose statistics are in s

  // The children of a node as bits.
  auto children = [&](int of) {
    return (uint64_t)__ballot_sync(0xFFFFFFFFu, s.parent[lane] == of) |
           (uint64_t)__ballot_sync(0xFFFFFFFFu, s.parent[lane + 32] == of) << 32;
  };
  // The statistics of `node`'s rows into pm, ps, qm, qs.  Where they are not
  // known, those of the nodes that follow it if every first child is accepted
  // are taken too, AHEAD in all: their rows are read together, and the cluster
  // meets once.
  auto enter = [&]() {
    if constexpr (!EAGER) {
      if (!(known >> node & 1)) {
        int count = 0;
        for (int at = node; at >= 0 && count < AHEAD;) {
          if (tid == 0) s.list[count] = at;
          ++count;
          known |= 1ull << at;
          const uint64_t next = children(at);
          at = next ? __ffsll((long long)next) - 1 : -1;
          if (at >= 0 && !children(at)) at = -1;  // a leaf's statistics have no use
        }
        __syncthreads();
        // The rows are dealt out to the warps; each takes its share of the
        // CTA's part of one of them.
        const int nrows = has_q ? 2 * count : count, per = WARPS / nrows;
        const int r = warp / per;
        if (r < nrows) {
          const int of = s.list[has_q ? r >> 1 : r];
          const E* row = has_q && (r & 1) ? draft + of * p.d_st : target + of * p.t_st;
          const int64_t groups = row_granules(p.V, (int)sizeof(E));
          const int g0 = (int)(groups * rank / cluster), g1 = (int)(groups * (rank + 1) / cluster);
          const MaxSum x = warp_join(row_share<DT, WALK_THREADS, WALK_DEPTH>(
              ring, row, vend, g0 + (warp - r * per) * 32 + lane, g1, per * 32, c));
          if (lane == 0) s.part[r][warp - r * per] = make_float2(x.m, x.s);
        }
        // (a value for each of the WARPS places of a row)
        if (lane < WARPS && lane >= per && warp < nrows) s.part[warp][lane] = make_float2(-INFINITY, 0.f);
        const float2 a = reduce(nrows, make_float2(-INFINITY, 0.f), [&](float2 x) {
          const MaxSum y = warp_join(MaxSum{x.x, x.y});
          return make_float2(y.m, y.s);
        });
        if (warp < nrows && lane == 0) {
          const int of = s.list[has_q ? warp >> 1 : warp];
          const bool q = has_q && (warp & 1);
          (q ? s.qm : s.pm)[of] = a.x == -INFINITY ? 0.f : a.x;
          (q ? s.qs : s.ps)[of] = a.y != 0.f ? 1.f / a.y : 0.f;
        }
        __syncthreads();
      }
    }
    pm = s.pm[node], ps = s.ps[node], qm = s.qm[node], qs = s.qs[node];
  };
  // P and Q of M consecutive entries from v after the node's first `count`
  // rejections, in the place of their scores.
  auto replay = [&](int v, int count, auto& P, auto& Q) {
    constexpr int M = sizeof(P) / sizeof(float);
#pragma unroll
    for (int e = 0; e < M; ++e) {
      P[e] = ex2(fmaf(P[e], c, -pm)) * ps;
      Q[e] = has_q ? ex2(fmaf(Q[e], c, -qm)) * qs : 0.f;
    }
    for (int i = 0; i < count; ++i) {
      const int hit = s.rx[i] - v;
      const float rz = s.rz[i], rzq = s.rzq[i];
#pragma unroll
      for (int e = 0; e < M; ++e) {
        const float left = has_q ? fmaxf(P[e] - Q[e], 0.f) : (hit == e ? 0.f : P[e]);
        if (rz > 0.f) P[e] = left * rz;
        Q[e] = hit == e ? 0.f : Q[e] * rzq;
      }
    }
  };
  // The thread's share of the vocabulary, a group of N entries at a time:
  // f(first entry, target scores, draft scores, noise).  Groups of 16 bytes go
  // through the ring, GROUP_DEPTH of them ahead.
  constexpr int SLOTS = 2 + N * 4 / 16;  // of a group: target, draft, noise
  constexpr int GROUP_DEPTH = WALK_DEPTH / (SLOTS > 3 ? 4 : 3);
  auto share = [&](const E* trow, const E* drow, const float* nrow, auto f) {
    if constexpr (N == 1) {
      constexpr int U = 4;
      for (int v = v0; v < vend; v += step * U) {
        float a[U][1], q[U][1], w[U][1];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (v + i * step < vend) {
            a[i][0] = score_at<DT>(trow, v + i * step);
            if (drow) q[i][0] = score_at<DT>(drow, v + i * step);
            if (nrow) w[i][0] = __ldg(nrow + v + i * step);
          }
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (v + i * step < vend) f(v + i * step, a[i], q[i], w[i]);
      }
    } else {
      Ring<WALK_THREADS, GROUP_DEPTH * SLOTS> in(ring), out(ring);
      constexpr uint32_t SLOT = WALK_THREADS * 16;
      int next = v0;
      const E *tp = trow + v0, *dp = drow + v0;
      const float* np = nrow + v0;
      auto issue = [&]() {
        if (next < vend) {
          cp_async16(in.at, tp, 16);
          if (drow) cp_async16(in.at + SLOT, dp, 16);
          if (nrow) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) cp_async16(in.at + (2 + i) * SLOT, np + 4 * i, 16);
          }
          next += step;
          tp += step, dp += step, np += step;
        }
        cp_async_commit();
        in.template next<SLOTS>();
      };
#pragma unroll
      for (int i = 0; i < GROUP_DEPTH - 1; ++i) issue();
      for (int v = v0; v < vend; v += step) {
        issue();
        cp_async_wait<GROUP_DEPTH - 1>();
        float a[N], q[N], w[N];
        ring_scores<DT, N>(out.at, a);
        if (drow) ring_scores<DT, N>(out.at + SLOT, q);
        if (nrow) {
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            float x[4];
            ring_scores<QMM_DT_F32, 4>(out.at + (2 + i) * SLOT, x);
            w[4 * i] = x[0], w[4 * i + 1] = x[1], w[4 * i + 2] = x[2], w[4 * i + 3] = x[3];
          }
        }
        f(v, a, q, w);
        out.template next<SLOTS>();
      }
      cp_async_wait<0>();
    }
  };
  uint64_t kids = children(node);
  if (kids) enter();
  while (kids) {
    const int child = __ffsll((long long)kids) - 1;
    kids &= kids - 1;
    const int x = s.token[child];
    float P[1] = {s.tx[child]}, Q[1] = {s.qx[child]};
    replay(x, rej, P, Q);
    if (s.u[child] * (has_q ? Q[0] : 1.f) < P[0]) {
      if (tid == 0) s.path[k] = child;
      ++k;
      node = child;
      // the next node's rejections overwrite this one's, which a slower warp may
      // still be reading above; a node whose statistics are known has no other barrier
      if (rej) __syncthreads();
      rej = 0;
      kids = children(node);
      if (kids) enter();
      continue;
    }
    if (kids) {
      // another sibling: Z and ZQ
      float z = 0.f, zq = 0.f;
      share(target + node * p.t_st, has_q ? draft + node * p.d_st : nullptr, nullptr,
            [&](int v, auto& a, auto& q, auto&) {
              replay(v, rej, a, q);
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const bool hit = v + e == x;
                z += has_q ? fmaxf(a[e] - q[e], 0.f) : (hit ? 0.f : a[e]);
                zq += hit ? 0.f : q[e];
              }
            });
      auto sum = [&](float2 y) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          y.x += __shfl_xor_sync(0xFFFFFFFFu, y.x, d);
          y.y += __shfl_xor_sync(0xFFFFFFFFu, y.y, d);
        }
        return y;
      };
      const float2 w = sum(make_float2(z, zq));
      if (lane == 0) s.part[0][warp] = w;
      const float2 t = reduce(1, make_float2(0.f, 0.f), sum);  // warp 0 holds it
      const float tz = t.x, tzq = t.y;
      if (tid == 0) {
        s.rz[rej] = tz > 0.f ? 1.f / tz : 0.f;
        s.rzq[rej] = tzq > 0.f ? 1.f / tzq : 1.f;
        s.rx[rej] = x;
      }
    } else if (tid == 0) {
      // the last child: only the race follows, and it needs no scale
      s.rz[rej] = 1.f;
      s.rzq[rej] = 1.f;
      s.rx[rej] = x;
    }
    ++rej;
    __syncthreads();
  }
  __syncthreads();

  // The next token: argmax P / noise.
  const E* trow = target + node * p.t_st;
  const E* drow = has_q ? draft + node * p.d_st : nullptr;
  constexpr int NONE = 0x7FFFFFFF;
  int token = 0;  // of thread 0
  if (rej == 0) {
    // Without a rejection entries are compared two at a time, by their scores'
    // difference and the noise's logarithms: a beats b where (a - b) c + log2(noise_b)
    // > log2(noise_a).  That needs no maximum of the row, which a node without
    // children has no other use for, and loses nothing to an offset of the scores.
    // The fast logarithm is off by 2^-22 at most near 1, less than three fp32
    // roundings of the race's values; -inf beats nothing (and a NaN neither).
    float top = -INFINITY, cost = 0.f;
    int at = NONE;  // a thread meets its entries in order: the first of equals stays
    share(trow, nullptr, noise, [&](int v, auto& a, auto&, auto& w) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float lw = __log2f(w[e]);
        if (fmaf(a[e] - top, c, cost) > lw) top = a[e], cost = lw, at = v + e;
      }
    });
    // of two candidates the one of the higher index has to beat the other, so that
    // both lanes of an exchange decide alike
    auto better = [&](float4 x) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        float4 o;
        o.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, d);
        o.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, d);
        o.z = __shfl_xor_sync(0xFFFFFFFFu, x.z, d);
        const bool late = __float_as_int(x.z) > __float_as_int(o.z);
        const float4 lo = late ? o : x, hi = late ? x : o;
        const bool beats = __float_as_int(hi.z) != NONE && fmaf(hi.x - lo.x, c, lo.y) > hi.y;
        x = beats ? hi : lo;
      }
      return x;
    };
    const float4 none = make_float4(-INFINITY, 0.f, __int_as_float(NONE), 0.f);
    const float4 x = better(make_float4(top, cost, __int_as_float(at), 0.f));
    if (lane == 0) reinterpret_cast<float4*>(s.part)[warp] = x;
    const float4 t = reduce(1, none, better);
    token = __float_as_int(t.z) == NONE ? 0 : __float_as_int(t.z);
  }
  // After a rejection P is there.  Where the last rejection leaves no mass, P stays
  // as it was before it: that, which rounding alone brings about, is another race.
  for (int undo = 0; rej > 0 && undo < 2; ++undo) {
    // a beats b where P_a noise_b > P_b noise_a; the quotient is taken once a thread
    // (for every entry it took 79 us instead of 70 for the batch above)
    float top = 0.f, cost = 1.f;
    int at = NONE;
    share(trow, drow, noise, [&](int v, auto& a, auto& q, auto& w) {
      replay(v, rej - 1, a, q);
      const int hit = s.rx[rej - 1] - v;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float pv = a[e];
        if (!undo) pv = has_q ? fmaxf(pv - q[e], 0.f) : (hit == e ? 0.f : pv);
        if (pv * cost > top * w[e]) top = pv, cost = w[e], at = v + e;
      }
    });
    // the largest quotient, which is positive, and the lowest index among equals, as
    // one 64-bit key; 0 for a thread with none
    const uint32_t key = __float_as_uint(top / cost);
    auto larger = [&](float2 x) {
      unsigned long long y = (unsigned long long)__float_as_uint(x.x) << 32 | __float_as_uint(x.y);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, y, d);
        y = o > y ? o : y;
      }
      return make_float2(__uint_as_float((uint32_t)(y >> 32)), __uint_as_float((uint32_t)y));
    };
    const float2 x = larger(at == NONE ? make_float2(0.f, 0.f)
                                       : make_float2(__uint_as_float(key), __uint_as_float(0xFFFFFFFFu - (uint32_t)at)));
    __syncthreads();
    if (lane == 0) s.part[0][warp] = x;
    const float2 t = reduce(1, make_float2(0.f, 0.f), larger);
    if (tid == 0) s.part[1][0] = t;
    __syncthreads();
    const uint32_t most = __float_as_uint(s.part[1][0].x), low = __float_as_uint(s.part[1][0].y);
    token = most ? (int)(0xFFFFFFFFu - low) : 0;
    if (most) break;  // something was left
  }
  if (rank == 0) {
    for (int i = tid; i < T; i += WALK_THREADS) p.path[(int64_t)b * T + i] = s.path[i];
    if (tid == 0) {
      p.accept[2 * b] = k;
      p.accept[2 * b + 1] = token;
    }
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// Parts of a row in the eager statistics: about four CTAs per SM; the most there are
// on any GPU.
int sample_chunks_most(int64_t V) {
  const int64_t most = (V + 4095) / 4096;
  return (int)(most < MAX_CHUNKS ? most : MAX_CHUNKS);
}
int sample_chunks(int B, int T, int64_t V, int sms) {
  const int64_t c = 4ll * sms / (2ll * B * (T > 1 ? T - 1 : 1));
  const int most = sample_chunks_most(V);
  return (int)(c < 1 ? 1 : (c > most ? most : c));
}
// CTAs of a walk: all that two on each SM allow, while each has two entries a
// thread and more.  Measured on 152 SMs, 151,936 entries of 16 bits, blocks of 16: with at
// most 152 / 304 / 608 CTAs 12 sequences took 45 / 42 / 42 us, 20 took 76 / 60 /
// 57, 32 took 78 / 70 / 81; 8 sequences of 1,000 entries 9.8 us, and 10.4 with
// clusters of 16.
int sample_cluster(int B, int64_t V, int sms) {
  int c = MAX_CLUSTER;
  while (c > 1 && ((int64_t)B * c > 2ll * sms || (int64_t)c * WALK_THREADS * 4 > 2 * V)) c /= 2;
  return c;
}
// Eager while reading the rows of all nodes costs less than the walk's own steps,
// one after the other, of the longest of its sequences: of a tree, or a long
// chain, most nodes are not visited, of a short chain they may all be.  Measured,
// eager against not, in us, 151,936 entries of 16 bits: 17 MB: 14 : 23; 34 MB: 21 :
// 26; chains of 8, 68 MB: 34 : 44; chains of 16, 109 MB: 37 : 42; 182 MB: 52 : 60;
// 292 MB: 71 : 70; chains of 32, 75 MB: 29 : 22; trees of 8, 85 MB: 38 : 34; of 16,
// 73 MB: 32 : 24; of 64 (50,257 entries of 32 bits), 101 MB: 28 : 13.  Chains of 17 to 31 were not measured.
bool sample_eager(int B, int T, int64_t V, int elem, bool has_q, bool chain) {
  const int64_t most = (chain && T <= 16 ? 192ll : 48ll) << 20;
  return T > 1 && (int64_t)B * (T - 1) * V * elem * (has_q ? 2 : 1) <= most;
}

template <int DT, bool WIDE, bool EAGER>
cudaError_t launch_walk(const SampleParams& p, int B, int cluster, cudaStream_t st) {
  auto kern = sample_walk_kernel<DT, WIDE, EAGER>;
  constexpr int SMEM = WALK_THREADS * WALK_DEPTH * 16;
  // once on each device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * cluster));
  cfg.blockDim = dim3(WALK_THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = EAGER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, cluster);
}

template <int DT, bool WIDE>
cudaError_t launch_sample(SampleParams& p, int B, int elem, int sms, cudaStream_t st) {
  const int cluster = sample_cluster(B, p.V, sms);
  if (!sample_eager(B, p.T, p.V, elem, p.draft != nullptr, p.parents == nullptr)) return launch_walk<DT, WIDE, false>(p, B, cluster, st);
  p.chunks = sample_chunks(B, p.T, p.V, sms);
  const int rows = (p.T - 1) * (p.draft ? 2 : 1);  // the last node has no children
  sample_stats_kernel<DT><<<dim3((unsigned)p.chunks, (unsigned)rows, (unsigned)B), STAT_THREADS,
                            STAT_THREADS * STAT_DEPTH * 16, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_walk<DT, WIDE, true>(p, B, cluster, st);
}

int check_sizes(int B, int T, int64_t V) {
  return B < 1 || B > 65535 || T < 1 || T > MAX_T || V < 1 || V > (1 << 24) ? QMM_ERR_SHAPE : QMM_OK;
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" {

int qmm_verify_sample_workspace(int B, int T, int64_t V, int64_t* bytes) {
  if (!bytes) return QMM_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check_sizes(B, T, V);
  if (rc != QMM_OK) return rc;
  // the most that any type, with or without drafter scores and parents, takes on any GPU
  *bytes = sample_eager(B, T, V, 2, false, true) ? (int64_t)B * T * 2 * sample_chunks_most(V) * (int64_t)sizeof(float2) : 256;
  return QMM_OK;
}

int qmm_verify_sample(const qmm_sample_args* a, void* stream) {
  if (!a || a->struct_size != sizeof(qmm_sample_args)) return QMM_ERR_INVALID_ARG;
  if (a->dtype > QMM_DT_F32) return QMM_ERR_INVALID_ARG;
  if (!a->target || !a->tokens || !a->u || !a->noise || !a->accept || !a->path || !a->workspace)
    return QMM_ERR_INVALID_ARG;
  int64_t need = 0;
  int rc = qmm_verify_sample_workspace(a->B, a->T, a->V, &need);
  if (rc != QMM_OK) return rc;
  if (a->workspace_bytes < need) return QMM_ERR_INVALID_ARG;
  const int elem = a->dtype == QMM_DT_F32 ? 4 : 2;
  if ((((uintptr_t)a->target | (uintptr_t)a->draft) & (elem - 1)) ||
      (((uintptr_t)a->tokens | (uintptr_t)a->parents | (uintptr_t)a->n_tokens | (uintptr_t)a->u |
        (uintptr_t)a->noise | (uintptr_t)a->temperature | (uintptr_t)a->accept | (uintptr_t)a->path) & 3) ||
      ((uintptr_t)a->workspace & 255))
    return QMM_ERR_ALIGN;
  int dev = 0, sms = 0;
  rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  SampleParams p;
  p.target = a->target;
  p.draft = a->draft;
  p.t_sb = a->target_stride[0], p.t_st = a->target_stride[1];
  p.d_sb = a->draft_stride[0], p.d_st = a->draft_stride[1];
  p.V = a->V;
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.n_tokens = a->n_tokens;
  p.u = a->u;
  p.noise = a->noise;
  p.temperature = a->temperature;
  p.accept = a->accept;
  p.path = a->path;
  p.stats = static_cast<float2*>(a->workspace);
  p.T = a->T;
  p.chunks = 1;
  // 16-byte loads where every row starts on a 16-byte boundary and holds whole
  // groups of them; single entries otherwise.
  const int64_t vec = 16 / elem;
  const bool wide = a->V % vec == 0 && a->V % 4 == 0 && !((uintptr_t)a->target & 15) && !((uintptr_t)a->noise & 15) &&
                    !(a->target_stride[0] % vec) && !(a->target_stride[1] % vec) &&
                    (!a->draft || (!((uintptr_t)a->draft & 15) && !(a->draft_stride[0] % vec) &&
                                   !(a->draft_stride[1] % vec)));
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  switch (a->dtype) {
    case QMM_DT_F32:
      e = wide ? launch_sample<QMM_DT_F32, true>(p, a->B, elem, sms, st) : launch_sample<QMM_DT_F32, false>(p, a->B, elem, sms, st);
      break;
    case QMM_DT_BF16:
      e = wide ? launch_sample<QMM_DT_BF16, true>(p, a->B, elem, sms, st) : launch_sample<QMM_DT_BF16, false>(p, a->B, elem, sms, st);
      break;
    default:
      e = wide ? launch_sample<QMM_DT_F16, true>(p, a->B, elem, sms, st) : launch_sample<QMM_DT_F16, false>(p, a->B, elem, sms, st);
  }
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

}  // extern "C"
