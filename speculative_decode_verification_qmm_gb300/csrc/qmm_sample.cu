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
// nodes only.  sample_eager() holds the rule.
#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {
namespace {

constexpr int MAX_T = QMM_TREE_MAX_T;
constexpr int STAT_THREADS = 256;
constexpr int WALK_THREADS = 512;
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_CHUNKS = 32;  // parts of a row in the eager statistics

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

// N consecutive scores from entry v: one 16-byte load, or one entry.
template <int DT, int N>
__device__ __forceinline__ void load_scores(const void* row, int64_t v, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = score_at<DT>(row, v);
  } else if constexpr (DT == QMM_DT_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + v));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + v));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = unpack16<DT == QMM_DT_BF16>((uint16_t)(w[i] & 0xFFFFu));
      x[2 * i + 1] = unpack16<DT == QMM_DT_BF16>((uint16_t)(w[i] >> 16));
    }
  }
}

template <int N>
__device__ __forceinline__ void load_noise(const float* row, int64_t v, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = __ldg(row + v);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + v + i));
      x[i] = a.x, x[i + 1] = a.y, x[i + 2] = a.z, x[i + 3] = a.w;
    }
  }
}

// Running (maximum, sum of 2^((x - maximum) c)) over a strided share of a row;
// the maximum is of the scores themselves.  c > 0.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  // a part whose maximum is -inf has no mass (its sum is 0, or NaN for NaN scores)
  r.s = (a.m == -INFINITY ? a.s : a.s * ex2((a.m - r.m) * c)) + (b.m == -INFINITY ? b.s : b.s * ex2((b.m - r.m) * c));
  return r;
}

template <int DT, int N>
__device__ __forceinline__ MaxSum row_share(const void* row, int64_t v0, int64_t v1, int64_t step, float c) {
  MaxSum a{-INFINITY, 0.f};
  constexpr int U = N == 1 ? 8 : 4;
  for (int64_t v = v0; v < v1; v += step * U) {
    float x[U][N];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (v + k * step < v1) {
        load_scores<DT, N>(row, v + k * step, x[k]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[k][e] = -INFINITY;
      }
    }
    float mx = a.m;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) mx = fmaxf(mx, x[k][e]);
    if (mx > a.m) {
      a.s = a.m == -INFINITY ? a.s : a.s * ex2((a.m - mx) * c);
      a.m = mx;
    }
    const float base = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) a.s += ex2((x[k][e] - base) * c);
  }
  return a;
}

__device__ __forceinline__ MaxSum warp_join(MaxSum a, float c) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    MaxSum o;
    o.m = __shfl_xor_sync(0xFFFFFFFFu, a.m, d);
    o.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, d);
    a = join(a, o, c);
  }
  return a;
}

__device__ __forceinline__ float log2e_over(const float* temperature, int b) {
  return 1.4426950408889634f / (temperature ? __ldg(temperature + b) : 1.f);
}

// ---------------------------------------------------------------- statistics
// CTA (chunk, row, sequence): (maximum, sum) of one part of row node = y / 2 of
// target (y even) or draft, if the node has children.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(STAT_THREADS) sample_stats_kernel(const __grid_constant__ SampleParams p) {
  constexpr int N = WIDE ? Score<DT>::VEC : 1;
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
  const int64_t groups = (p.V + N - 1) / N;
  const int64_t g0 = groups * blockIdx.x / p.chunks, g1 = groups * (blockIdx.x + 1) / p.chunks;
  MaxSum a = row_share<DT, N>(row, (g0 + tid) * N, g1 * N, (int64_t)STAT_THREADS * N, c);
  a = warp_join(a, c);
  if ((tid & 31) == 0) s_part[tid >> 5] = a;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < STAT_THREADS / 32; ++w) a = join(a, s_part[w], c);
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
  float4 part[WALK_THREADS / 32];    // per warp
  unsigned long long best[WALK_THREADS / 32];
  float4 cl[2];                      // this CTA's part of a cluster sum, two in turn
  unsigned long long cl_best;
};

template <int DT, bool WIDE, bool EAGER>
__global__ void __launch_bounds__(WALK_THREADS, 2) sample_walk_kernel(const __grid_constant__ SampleParams p,
                                                                   int cluster) {
  constexpr int N = WIDE ? Score<DT>::VEC : 1;
  using E = typename Score<DT>::type;
  __shared__ WalkSmem s;
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
      a = warp_join(a, c);
      if (lane == 0) {
        (side ? s.qm : s.pm)[node] = a.m == -INFINITY ? 0.f : a.m;
        (side ? s.qs : s.ps)[node] = a.s != 0.f ? 1.f / a.s : 0.f;
      }
    }
  }
  __syncthreads();

  int turn = 0;
  // Thread 0's value of every CTA of the cluster: lane r of each warp gets
  // rank r's, the other lanes `none`.
  auto exchange = [&](float4 mine, float4 none) {
    if (tid == 0) s.cl[turn] = mine;
    cluster_sync_all();
    if (lane < cluster) {
      const uint32_t a = dsmem_map(smem_u32(&s.cl[turn]), lane);
      none = make_float4(ld_dsmem_f32(a), ld_dsmem_f32(a + 4), ld_dsmem_f32(a + 8), ld_dsmem_f32(a + 12));
    }
    turn ^= 1;
    return none;
  };

  const int64_t v0 = ((int64_t)rank * WALK_THREADS + tid) * N;
  const int64_t step = (int64_t)cluster * WALK_THREADS * N;
  const int64_t vend = p.V;

  int node = 0, k = 0, rej = 0;
  float pm = 0.f, ps = 0.f, qm = 0.f, qs = 0.f;

  // The statistics of `node`'s rows into pm, ps, qm, qs.
  auto enter = [&](bool need) {
    if constexpr (EAGER) {
      pm = s.pm[node], ps = s.ps[node], qm = s.qm[node], qs = s.qs[node];
    } else if (need) {
      MaxSum a = row_share<DT, N>(target + node * p.t_st, v0, vend, step, c);
      MaxSum q{-INFINITY, 0.f};
      if (has_q) q = row_share<DT, N>(draft + node * p.d_st, v0, vend, step, c);
      a = warp_join(a, c);
      q = warp_join(q, c);
      if (lane == 0) s.part[warp] = make_float4(a.m, a.s, q.m, q.s);
      __syncthreads();
      if (tid == 0)
        for (int w = 1; w < WALK_THREADS / 32; ++w) {
          const float4 o = s.part[w];
          a = join(a, MaxSum{o.x, o.y}, c);
          q = join(q, MaxSum{o.z, o.w}, c);
        }
      const float4 o = exchange(make_float4(a.m, a.s, q.m, q.s), make_float4(-INFINITY, 0.f, -INFINITY, 0.f));
      const MaxSum ta = warp_join(MaxSum{o.x, o.y}, c), tq = warp_join(MaxSum{o.z, o.w}, c);
      pm = ta.m == -INFINITY ? 0.f : ta.m;
      ps = ta.s != 0.f ? 1.f / ta.s : 0.f;
      qm = tq.m == -INFINITY ? 0.f : tq.m;
      qs = tq.s != 0.f ? 1.f / tq.s : 0.f;
    }
  };
  // P and Q of entry v after the node's rejections, from their values before any.
  auto replay = [&](int v, float& P, float& Q) {
    for (int i = 0; i < rej; ++i) {
      const bool hit = v == s.rx[i];
      const float left = has_q ? fmaxf(P - Q, 0.f) : (hit ? 0.f : P);
      if (s.rz[i] > 0.f) P = left * s.rz[i];
      Q = hit ? 0.f : Q * s.rzq[i];
    }
  };
  // The children of `node` as bits.
  auto children = [&]() {
    return (uint64_t)__ballot_sync(0xFFFFFFFFu, s.parent[lane] == node) |
           (uint64_t)__ballot_sync(0xFFFFFFFFu, s.parent[lane + 32] == node) << 32;
  };

  uint64_t kids = children();
  enter(kids != 0);
  while (kids) {
    const int child = __ffsll((long long)kids) - 1;
    kids &= kids - 1;
    const int x = s.token[child];
    float P = ex2((s.tx[child] - pm) * c) * ps;
    float Q = has_q ? ex2((s.qx[child] - qm) * c) * qs : 0.f;
    replay(x, P, Q);
    if (s.u[child] * (has_q ? Q : 1.f) < P) {
      if (tid == 0) s.path[k] = child;
      ++k;
      node = child;
      rej = 0;
      kids = children();
      enter(kids != 0);
      continue;
    }
    if (kids) {
      // another sibling: Z and ZQ
      float z = 0.f, zq = 0.f;
      const E* trow = target + node * p.t_st;
      const E* drow = draft + node * p.d_st;
      for (int64_t v = v0; v < vend; v += step) {
        float a[N], q[N];
        load_scores<DT, N>(trow, v, a);
        if (has_q) load_scores<DT, N>(drow, v, q);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float pv = ex2((a[e] - pm) * c) * ps;
          float qv = has_q ? ex2((q[e] - qm) * c) * qs : 0.f;
          replay((int)v + e, pv, qv);
          const bool hit = (int)v + e == x;
          z += has_q ? fmaxf(pv - qv, 0.f) : (hit ? 0.f : pv);
          zq += hit ? 0.f : qv;
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
        zq += __shfl_xor_sync(0xFFFFFFFFu, zq, d);
      }
      if (lane == 0) s.part[warp] = make_float4(z, zq, 0.f, 0.f);
      __syncthreads();
      if (tid == 0)
        for (int w = 1; w < WALK_THREADS / 32; ++w) {
          z += s.part[w].x;
          zq += s.part[w].y;
        }
      const float4 o = exchange(make_float4(z, zq, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f));
      float tz = o.x, tzq = o.y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        tz += __shfl_xor_sync(0xFFFFFFFFu, tz, d);
        tzq += __shfl_xor_sync(0xFFFFFFFFu, tzq, d);
      }
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

  // The next token: argmax P / noise.  Where the last rejection leaves no mass,
  // P stays as it was before it: both are raced, and the second counts then.
  // Without a rejection the race is run on logarithms, (score / temperature)
  // log2(e) - log2(noise): they need no maximum of the row, which a node
  // without children has no other use for.
  unsigned long long best = 0, kept = 0;
  auto race = [](unsigned long long& to, float r, int v) {
    if (r != r) return;
    uint32_t o = __float_as_uint(r);
    o = o & 0x80000000u ? ~o : o | 0x80000000u;  // the order of the values
    const unsigned long long key = (unsigned long long)o << 32 | (0xFFFFFFFFu - (uint32_t)v);
    to = key > to ? key : to;
  };
  const E* trow = target + node * p.t_st;
  const E* drow = draft + node * p.d_st;
  if (rej == 0) {
    constexpr int U = N == 1 ? 8 : 2;
    for (int64_t v = v0; v < vend; v += step * U) {
      float a[U][N], w[U][N];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + i * step < vend) {
          load_scores<DT, N>(trow, v + i * step, a[i]);
          load_noise<N>(noise, v + i * step, w[i]);
        }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + i * step < vend) {
#pragma unroll
          for (int e = 0; e < N; ++e) race(best, fmaf(a[i][e], c, -__log2f(w[i][e])), (int)(v + i * step) + e);
        }
    }
  } else {
    for (int64_t v = v0; v < vend; v += step) {
      float a[N], q[N], w[N];
      load_scores<DT, N>(trow, v, a);
      if (has_q) load_scores<DT, N>(drow, v, q);
      load_noise<N>(noise, v, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int vi = (int)v + e;
        float pv = ex2((a[e] - pm) * c) * ps;
        float qv = has_q ? ex2((q[e] - qm) * c) * qs : 0.f;
        for (int i = 0; i < rej - 1; ++i) {
          const bool hit = vi == s.rx[i];
          const float left = has_q ? fmaxf(pv - qv, 0.f) : (hit ? 0.f : pv);
          if (s.rz[i] > 0.f) pv = left * s.rz[i];
          qv = hit ? 0.f : qv * s.rzq[i];
        }
        race(kept, __fdiv_rn(pv, w[e]), vi);
        race(best, __fdiv_rn(has_q ? fmaxf(pv - qv, 0.f) : (vi == s.rx[rej - 1] ? 0.f : pv), w[e]), vi);
      }
    }
  }
  auto block_max = [&](unsigned long long key) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
      key = o > key ? o : key;
    }
    __syncthreads();
    if (lane == 0) s.best[warp] = key;
    __syncthreads();
    for (int w = 0; w < WALK_THREADS / 32; ++w) key = s.best[w] > key ? s.best[w] : key;
    return key;
  };
  best = block_max(best);
  kept = rej > 0 ? block_max(kept) : 0;
  {
    const float4 o = exchange(make_float4(__uint_as_float((uint32_t)(best >> 32)), __uint_as_float((uint32_t)best),
                                          __uint_as_float((uint32_t)(kept >> 32)), __uint_as_float((uint32_t)kept)),
                              make_float4(0.f, 0.f, 0.f, 0.f));
    best = (unsigned long long)__float_as_uint(o.x) << 32 | __float_as_uint(o.y);
    kept = (unsigned long long)__float_as_uint(o.z) << 32 | __float_as_uint(o.w);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long x = __shfl_xor_sync(0xFFFFFFFFu, best, d), y = __shfl_xor_sync(0xFFFFFFFFu, kept, d);
      best = x > best ? x : best;
      kept = y > kept ? y : kept;
    }
  }
  if (rej > 0 && (uint32_t)(best >> 32) <= 0x80000000u) best = kept;  // nothing was left
  if (rank == 0) {
    for (int i = tid; i < T; i += WALK_THREADS) p.path[(int64_t)b * T + i] = s.path[i];
    if (tid == 0) {
      p.accept[2 * b] = k;
      p.accept[2 * b + 1] = best ? (int)(0xFFFFFFFFu - (uint32_t)best) : 0;
    }
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// Parts of a row in the eager statistics, and CTAs of a walk.
int sample_chunks(int B, int T, int64_t V) {
  int64_t c = 608 / (2ll * B * (T > 1 ? T - 1 : 1));  // about four CTAs per SM
  const int64_t most = (V + 4095) / 4096;
  c = c < most ? c : most;
  return (int)(c < 1 ? 1 : (c > MAX_CHUNKS ? MAX_CHUNKS : c));
}
int sample_cluster(int B, int64_t V) {
  int c = MAX_CLUSTER;
  while (c > 1 && ((int64_t)B * c > 304 || (int64_t)c * WALK_THREADS * 4 > 2 * V)) c /= 2;
  return c;
}
// Eager while the rows of all nodes are read in about the time of one step of
// the walk.
bool sample_eager(int B, int T, int64_t V, int elem, bool has_q) {
  return T > 1 && (int64_t)B * (T - 1) * V * elem * (has_q ? 2 : 1) <= (32ll << 20);
}

template <int DT, bool WIDE, bool EAGER>
cudaError_t launch_walk(const SampleParams& p, int B, int cluster, cudaStream_t st) {
  auto kern = sample_walk_kernel<DT, WIDE, EAGER>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * cluster));
  cfg.blockDim = dim3(WALK_THREADS);
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
cudaError_t launch_sample(SampleParams& p, int B, int elem, cudaStream_t st) {
  const int cluster = sample_cluster(B, p.V);
  if (!sample_eager(B, p.T, p.V, elem, p.draft != nullptr)) return launch_walk<DT, WIDE, false>(p, B, cluster, st);
  p.chunks = sample_chunks(B, p.T, p.V);
  const int rows = (p.T - 1) * (p.draft ? 2 : 1);  // the last node has no children
  sample_stats_kernel<DT, WIDE><<<dim3((unsigned)p.chunks, (unsigned)rows, (unsigned)B), STAT_THREADS, 0, st>>>(p);
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
  *bytes = sample_eager(B, T, V, 2, false) ? (int64_t)B * T * 2 * sample_chunks(B, T, V) * (int64_t)sizeof(float2) : 256;
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
      e = wide ? launch_sample<QMM_DT_F32, true>(p, a->B, elem, st) : launch_sample<QMM_DT_F32, false>(p, a->B, elem, st);
      break;
    case QMM_DT_BF16:
      e = wide ? launch_sample<QMM_DT_BF16, true>(p, a->B, elem, st) : launch_sample<QMM_DT_BF16, false>(p, a->B, elem, st);
      break;
    default:
      e = wide ? launch_sample<QMM_DT_F16, true>(p, a->B, elem, st) : launch_sample<QMM_DT_F16, false>(p, a->B, elem, st);
  }
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

}  // extern "C"
