// qmm_scores.cu -- penalties, biases and grammar masks on the scores of a drafted
// tree (qmm_adjust_scores in include/qmm.h), and the counts that they go by
// (qmm_count_tokens).
//
// Mathematics.  With c(v) the times that token v was emitted, the node's own path
// included: x -> x / r (x > 0) or x r where v was seen; x - f c - p [c > 0] + bias; -inf
// where the grammar bit is 0.
//
// A CTA takes a range of the vocabulary of one sequence and walks its nodes, the scores of
// AHEAD of them in flight: the counts, prompt bits and biases of the range are read once, for
// all nodes, as two factors and a term for each entry.  Which nodes lie on a node's path
// is one bit each of a 64-bit word; where a node's tokens fall into the range, which few
// do, their entries are worked out anew.
// What bounds it: memory for large batches (32 chains of 16 x 151,936, bf16, with biases and masks 73.6 us,
// 4.6 TB/s, 69 % of a copy; without them 68.4 and 4.8, trees 65.0 and 5.1), a launch and two dependent
// loads for one tree (8 x 151,936, fp32: 4.7 us); rows that do not begin on 16 bytes are bound by the number
// of loads and stores, one an entry (32 x 16 x 50,257, bf16: 38 us, of 50,256 29.5).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {
namespace {

constexpr int MAX_T = QMM_TREE_MAX_T;
constexpr int THREADS = 256;
constexpr int E = 8;  // entries of a thread
constexpr int RANGE = THREADS * E;
constexpr int CTAS_PER_SM = 4;

struct AdjustParams {
  const void* scores;
  void* out;
  int64_t s_sb, s_st, o_sb, o_st;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* n_tokens;
  const int32_t* counts;
  const uint32_t* prompt;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const float* bias;
  const uint32_t* mask;
  int64_t ld_counts, ld_prompt, ld_bias, m_sb, m_st;
  int64_t V;
  int T;
  int per;  // nodes of a CTA
};

// Entry e of thread t lies at the range's place(e, t): 8 side by side, or every 32nd of a
// warp's 256, for which no alignment is needed.
template <bool WIDE>
__device__ __forceinline__ int place(int e, int t) {
  return WIDE ? t * E + e : (t >> 5) * 32 * E + e * 32 + (t & 31);
}

// A thread's eight scores as they are in memory (fp32: 8 words, else 4), and their values.
// `mine` is where its first entry lies, `left` how many entries there are from it on.
template <int DT>
struct Raw {
  static constexpr int WORDS = DT == QMM_DT_F32 ? 8 : 4;
  uint32_t w[WORDS];
};

template <int DT, bool WIDE>
__device__ __forceinline__ void load8(const char* mine, int left, Raw<DT>& r) {
  if constexpr (WIDE) {
    const uint4* p = reinterpret_cast<const uint4*>(mine);
#pragma unroll
    for (int i = 0; i < Raw<DT>::WORDS / 4; ++i) {
      const uint4 v = i * 4 < left ? __ldcs(p + i) : make_uint4(0u, 0u, 0u, 0u);
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else {
    auto get = [&](auto whole) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = decltype(whole)::value || 32 * e < left;
        if constexpr (DT == QMM_DT_F32) {
          r.w[e] = in ? __ldcs(reinterpret_cast<const uint32_t*>(mine) + 32 * e) : 0u;
        } else {
          const uint32_t x = in ? __ldcs(reinterpret_cast<const uint16_t*>(mine) + 32 * e) : 0;
          r.w[e / 2] = e & 1 ? r.w[e / 2] | x << 16 : x;
        }
      }
    };
    if (left > 32 * (E - 1))
      get(std::true_type());
    else
      get(std::false_type());
  }
}

template <int DT>
__device__ __forceinline__ void values(const Raw<DT>& r, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (DT == QMM_DT_F32)
      x[e] = __uint_as_float(r.w[e]);
    else
      x[e] = unpack16<DT == QMM_DT_BF16>((uint16_t)(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2]));
  }
}

template <int DT, bool WIDE>
__device__ __forceinline__ void store8(char* mine, int left, const float (&x)[E]) {
  if constexpr (WIDE && DT == QMM_DT_F32) {
    float4* p = reinterpret_cast<float4*>(mine);
    if (left > 0) __stcs(p, make_float4(x[0], x[1], x[2], x[3]));
    if (left > 4) __stcs(p + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else if constexpr (WIDE) {
    constexpr bool BF = DT == QMM_DT_BF16;
    if (left > 0)
      __stcs(reinterpret_cast<uint4*>(mine),
             make_uint4(pack16<BF>(x[0], x[1]), pack16<BF>(x[2], x[3]), pack16<BF>(x[4], x[5]), pack16<BF>(x[6], x[7])));
  } else {
    auto put = [&](auto whole) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!decltype(whole)::value && 32 * e >= left) continue;
        if constexpr (DT == QMM_DT_F32)
          __stcs(reinterpret_cast<float*>(mine) + 32 * e, x[e]);
        else
          __stcs(reinterpret_cast<uint16_t*>(mine) + 32 * e, (uint16_t)pack16<DT == QMM_DT_BF16>(x[e], 0.f));
      }
    };
    if (left > 32 * (E - 1))
      put(std::true_type());
    else
      put(std::false_type());
  }
}

// The bits of a thread's eight entries, from the word that it loaded (a range is whole
// words): WIDE, a byte of it; else lane e has the word of the warp's entries e.
template <bool WIDE>
__device__ __forceinline__ uint32_t bits_of(uint32_t loaded) {
  if constexpr (WIDE) return loaded >> (8 * (threadIdx.x & 3)) & 255u;
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) r |= (__shfl_sync(0xFFFFFFFFu, loaded, e) >> (threadIdx.x & 31) & 1u) << e;
  return r;
}

template <int DT, bool WIDE, int AHEAD>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) adjust_kernel(const __grid_constant__ AdjustParams p) {
  __shared__ int s_token[MAX_T];                // place in the range
  __shared__ unsigned long long s_path[MAX_T];  // the nodes of a node's path whose tokens lie in the range
  __shared__ int s_up[MAX_T];
  const int t = threadIdx.x, b = blockIdx.y;
  const int64_t v0 = (int64_t)blockIdx.x * RANGE, left = p.V - v0;
  int n = p.T;
  if (p.n_tokens) {
    n = __ldg(p.n_tokens + b);
    n = n < 0 ? 0 : (n > p.T ? p.T : n);
  }
  const int first = blockIdx.z * p.per, end = first + p.per < n ? first + p.per : n;
  if (first >= end) return;
  const bool penal = p.repetition || p.frequency || p.presence;
  float c[E], bias[E];
  uint32_t asked = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = 0.f, bias[e] = 0.f;
  // what this thread has of each row, and of its bits
  constexpr int ELEM = DT == QMM_DT_F32 ? 4 : 2;
  const int own = place<WIDE>(0, t);
  const int have = left - own > RANGE ? RANGE : (left - own < 0 ? 0 : (int)(left - own));
  const char* src = static_cast<const char*>(p.scores) + (b * p.s_sb + first * p.s_st + v0 + own) * ELEM;
  char* dst = static_cast<char*>(p.out) + (b * p.o_sb + first * p.o_st + v0 + own) * ELEM;
  const int64_t src_step = p.s_st * ELEM, dst_step = p.o_st * ELEM;
  const int word = WIDE ? t / 4 : (t >> 5) * E + (t & 31);
  const bool has_word = (WIDE || (t & 31) < E) && word * 32 < left;
  const uint32_t* mask = p.mask ? p.mask + b * p.m_sb + first * p.m_st + v0 / 32 + word : nullptr;
  // the first nodes' scores and bits are on their way while the rest is looked up
  Raw<DT> raw[AHEAD];
  uint32_t may[AHEAD];
  auto request = [&](int i0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (i0 + k >= end) continue;
      load8<DT, WIDE>(src, have, raw[k]);
      src += src_step;
      if (mask) {
        may[k] = has_word ? __ldg(mask) : 0u;
        mask += p.m_st;
      }
    }
  };
  request(first);
  float rep = 1.f, inv = 1.f, freq = 0.f, pres = 0.f;
  bool paths = false;
  if (penal) {
    if (p.repetition) rep = __ldg(p.repetition + b), inv = 1.f / rep;
    if (p.frequency) freq = __ldg(p.frequency + b);
    if (p.presence) pres = __ldg(p.presence + b);
    if (p.counts) {
      const int32_t* row = p.counts + b * p.ld_counts + v0;
      if constexpr (WIDE) {
        const int4* q = reinterpret_cast<const int4*>(row + t * E);
        const int4 u = t * E < left ? __ldg(q) : make_int4(0, 0, 0, 0), w = t * E + 4 < left ? __ldg(q + 1) : make_int4(0, 0, 0, 0);
        c[0] = (float)u.x, c[1] = (float)u.y, c[2] = (float)u.z, c[3] = (float)u.w;
        c[4] = (float)w.x, c[5] = (float)w.y, c[6] = (float)w.z, c[7] = (float)w.w;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) c[e] = place<false>(e, t) < left ? (float)__ldg(row + place<false>(e, t)) : 0.f;
      }
    }
    if (p.prompt && has_word) asked = __ldg(p.prompt + b * p.ld_prompt + v0 / 32 + word);
    int64_t x = -1;
    if (t < n && p.tokens) x = __ldg(p.tokens + (int64_t)b * p.T + t) - v0;
    const bool here = t > 0 && t < n && x >= 0 && x < RANGE && x < left;
    // (mostly no node's token falls into the range)
    paths = __syncthreads_or(here);
    if (paths) {
      // A path is the nodes' own bits and the parent's path: each round doubles how far it
      // reaches.  What does not come before its node ends it.
      if (t < MAX_T) {
        int up = 0;
        if (t > 0 && t < n) up = p.parents ? __ldg(p.parents + (int64_t)b * p.T + t) : t - 1;
        s_up[t] = up > 0 && up < t ? up : 0;
        s_path[t] = here ? 1ull << t : 0;
        s_token[t] = here ? (int)x : -1;
      }
      for (int reach = 1; reach < n; reach *= 2) {
        __syncthreads();
        unsigned long long path = 0;
        int up = 0;
        if (t < MAX_T) path = s_path[t] | s_path[s_up[t]], up = s_up[s_up[t]];
        __syncthreads();
        if (t < MAX_T) s_path[t] = path, s_up[t] = up;
      }
      __syncthreads();
    }
  }
  if (p.bias) {
    const float* row = p.bias + b * p.ld_bias + v0;
    if constexpr (WIDE) {
      const float4* q = reinterpret_cast<const float4*>(row + t * E);
      const float4 u = t * E < left ? __ldg(q) : make_float4(0.f, 0.f, 0.f, 0.f),
                   w = t * E + 4 < left ? __ldg(q + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      bias[0] = u.x, bias[1] = u.y, bias[2] = u.z, bias[3] = u.w, bias[4] = w.x, bias[5] = w.y, bias[6] = w.z, bias[7] = w.w;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) bias[e] = place<false>(e, t) < left ? __ldg(row + place<false>(e, t)) : 0.f;
    }
  }
  // An entry becomes x (up for x > 0, else down) - term.  (The inverse costs one rounding of fp32 more
  // than a division, which took 77 to 112 us instead of 65 for 32 x 16 x 151,936, bf16, as more
  // entries were seen.)
  const uint32_t in_prompt = bits_of<WIDE>(asked);
  float up[E], down[E], term[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool seen = c[e] > 0.f || (in_prompt >> e & 1);
    up[e] = seen ? inv : 1.f;
    down[e] = seen ? rep : 1.f;
    term[e] = freq * c[e] + (c[e] > 0.f ? pres : 0.f) - bias[e];
  }
  for (int i0 = first; i0 < end; i0 += AHEAD) {
    if (i0 > first) request(i0);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k;
      if (i >= end) continue;
      float x[E], y[E];
      values<DT>(raw[k], x);
      const uint32_t bits = mask ? bits_of<WIDE>(may[k]) : 255u;
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = fmaf(x[e], x[e] > 0.f ? up[e] : down[e], -term[e]);
      const unsigned long long path = paths ? s_path[i] : 0;
      if (path) {
        uint64_t more = 0;  // how often each entry is on the path, in bytes
        for (unsigned long long rest = path; rest; rest &= rest - 1) {
          const int at = s_token[__ffsll((long long)rest) - 1];
          const int owner = WIDE ? at / E : (at / (32 * E)) * 32 + at % 32, e = WIDE ? at % E : at / 32 % E;
          if (owner == t) more += 1ull << (8 * e);
        }
        if (more) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int again = (int)(more >> (8 * e)) & 255;
            if (!again) continue;
            // (what it was emitted before is not kept in registers for this)
            const int64_t v = v0 + place<WIDE>(e, t);
            const float k = (float)(again + (p.counts ? __ldg(p.counts + b * p.ld_counts + v) : 0));
            const float add = p.bias ? __ldg(p.bias + b * p.ld_bias + v) : 0.f;
            y[e] = fmaf(x[e], x[e] > 0.f ? inv : rep, add - (freq * k + pres));
          }
        }
      }
      if (mask) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = bits >> e & 1 ? y[e] : -INFINITY;
      }
      store8<DT, WIDE>(dst, have, y);
      dst += dst_step;
    }
  }
}

template <int DT>
cudaError_t launch_adjust(const AdjustParams& p, int B, bool wide, int sms, cudaStream_t st) {
  AdjustParams q = p;
  const int64_t ranges = (p.V + RANGE - 1) / RANGE, ctas = ranges * B, slots = (int64_t)CTAS_PER_SM * sms;
  // How many CTAs share a sequence's nodes: what takes the fewest nodes one after another,
  // where a CTA begins as long as two nodes take.  (32 x 16 nodes of 50,256, bf16: 31.3 us by one CTA, in two
  // waves the second of which is a third full, 27.4 by two, in three waves; 8 x 16 of 50,257, fp32: 16.3
  // by four, 15.6 by six; 64 nodes of 50,256: 9.9 by 22 in one wave, 11.2 by 32 in two.)
  int64_t best = INT64_MAX;
  for (int per = 1; per <= p.T; ++per) {
    const int64_t cost = (ctas * ((p.T + per - 1) / per) + slots - 1) / slots * (per + 2);
    if (cost <= best) best = cost, q.per = per;
  }
  const dim3 grid((unsigned)ranges, (unsigned)B, (unsigned)((p.T + q.per - 1) / q.per));
  // Two nodes in flight, but for a CTA's only node, and where entries are loaded one by one, which
  // keeps enough in flight.  (One : two, us: 32 x 16 nodes of 151,936, bf16, 74 : 66; 8 nodes of
  // 151,936, one a CTA, 4.5 : 5.0; 32 x 16 of 50,257, bf16, 36 : 38.)
  if (wide && q.per > 1)
    adjust_kernel<DT, true, 2><<<grid, THREADS, 0, st>>>(q);
  else if (wide)
    adjust_kernel<DT, true, 1><<<grid, THREADS, 0, st>>>(q);
  else
    adjust_kernel<DT, false, 1><<<grid, THREADS, 0, st>>>(q);
  return cudaGetLastError();
}

__global__ void count_kernel(int32_t* counts, int64_t ld, int T, int64_t V, const int32_t* tokens, const int32_t* path,
                             const int32_t* accept) {
  const int b = blockIdx.x, j = threadIdx.x;
  const int k = __ldg(accept + 2 * b);
  int x = -1;
  if (j < T && j < k) {
    const int node = __ldg(path + (int64_t)b * T + j);
    if (node >= 0 && node < T) x = __ldg(tokens + (int64_t)b * T + node);
  } else if (j == MAX_T) {
    x = __ldg(accept + 2 * b + 1);
  }
  if (x >= 0 && x < V) atomicAdd(counts + b * ld + x, 1);
}

int check_sizes(int B, int T, int64_t V) {
  return B < 1 || B > 65535 || T < 1 || T > MAX_T || V < 1 || V > (1 << 24) ? QMM_ERR_SHAPE : QMM_OK;
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" {

int qmm_adjust_scores(const qmm_adjust_args* a, void* stream) {
  if (!a || a->struct_size != sizeof(qmm_adjust_args)) return QMM_ERR_INVALID_ARG;
  if (a->dtype > QMM_DT_F32 || !a->scores || !a->out) return QMM_ERR_INVALID_ARG;
  int rc = check_sizes(a->B, a->T, a->V);
  if (rc != QMM_OK) return rc;
  const int64_t words = (a->V + 31) / 32;
  const int elem = a->dtype == QMM_DT_F32 ? 4 : 2;
  const uintptr_t small = (uintptr_t)a->tokens | (uintptr_t)a->parents | (uintptr_t)a->n_tokens | (uintptr_t)a->counts |
                          (uintptr_t)a->prompt | (uintptr_t)a->repetition | (uintptr_t)a->frequency |
                          (uintptr_t)a->presence | (uintptr_t)a->bias | (uintptr_t)a->mask;
  if ((((uintptr_t)a->scores | (uintptr_t)a->out) & (elem - 1)) || (small & 3)) return QMM_ERR_ALIGN;
  if (a->B > 1 && ((a->counts && a->ld_counts < a->V) || (a->prompt && a->ld_prompt < words) ||
                   (a->bias && a->ld_bias && a->ld_bias < a->V)))
    return QMM_ERR_ALIGN;
  AdjustParams p;
  // strides of dimensions with one entry are not followed
  const bool bs = a->B > 1, ts = a->T > 1;
  p.s_sb = bs ? a->stride[0] : 0, p.s_st = ts ? a->stride[1] : 0;
  p.o_sb = bs ? a->out_stride[0] : 0, p.o_st = ts ? a->out_stride[1] : 0;
  p.m_sb = bs ? a->mask_stride[0] : 0, p.m_st = ts ? a->mask_stride[1] : 0;
  if (a->out == a->scores && (p.s_sb != p.o_sb || p.s_st != p.o_st)) return QMM_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  p.scores = a->scores, p.out = a->out;
  p.tokens = a->tokens, p.parents = a->parents, p.n_tokens = a->n_tokens;
  p.counts = a->counts, p.prompt = a->prompt;
  p.repetition = a->repetition, p.frequency = a->frequency, p.presence = a->presence;
  p.bias = a->bias, p.mask = a->mask;
  p.ld_counts = bs ? a->ld_counts : 0, p.ld_prompt = bs ? a->ld_prompt : 0, p.ld_bias = bs ? a->ld_bias : 0;
  p.V = a->V;
  p.T = a->T;
  p.per = a->T;
  // 16-byte loads where every row of every tensor starts on a boundary and holds
  // whole groups of eight scores (and so of eight bits)
  const bool wide = !((a->V | p.s_sb | p.s_st | p.o_sb | p.o_st) & 7) && !(((uintptr_t)a->scores | (uintptr_t)a->out) & 15) &&
                    !(a->counts && (((uintptr_t)a->counts & 15) || (p.ld_counts & 3))) &&
                    !(a->bias && (((uintptr_t)a->bias & 15) || (p.ld_bias & 3)));
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  switch (a->dtype) {
    case QMM_DT_F32: e = launch_adjust<QMM_DT_F32>(p, a->B, wide, sms, st); break;
    case QMM_DT_BF16: e = launch_adjust<QMM_DT_BF16>(p, a->B, wide, sms, st); break;
    default: e = launch_adjust<QMM_DT_F16>(p, a->B, wide, sms, st); break;
  }
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

int qmm_count_tokens(int32_t* counts, int64_t ld_counts, int B, int T, int64_t V, const int32_t* tokens,
                     const int32_t* path, const int32_t* accept, void* stream) {
  if (!counts || !tokens || !path || !accept) return QMM_ERR_INVALID_ARG;
  int rc = check_sizes(B, T, V);
  if (rc != QMM_OK) return rc;
  if ((((uintptr_t)counts | (uintptr_t)tokens | (uintptr_t)path | (uintptr_t)accept) & 3) || (B > 1 && ld_counts < V))
    return QMM_ERR_ALIGN;
  int dev = 0, sms = 0;
  rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  count_kernel<<<B, MAX_T + 32, 0, (cudaStream_t)stream>>>(counts, ld_counts, T, V, tokens, path, accept);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

}  // extern "C"
