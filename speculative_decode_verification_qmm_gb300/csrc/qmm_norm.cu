// qmm_norm.cu -- residual sums with the norms before and after a block
// (qmm_residual_norm in include/qmm.h).
//
// Mathematics.  z = y or norm(y) w_p + b_p;  r' = r + s g z;  out = norm(r') w + b,
// norm(x) = x rsqrt(mean x^2 + eps), or of x - mean x: the mean first, then the mean
// square of the differences, which does not cancel.
//
// Rows of up to SHORT entries: a warp each, straight from memory.  Longer ones: a CTA each,
// which holds a whole row in registers, E entries a thread, so that r' is normalised
// unrounded; the inputs of its next rows are on their way into shared memory meanwhile.
// They are copied in groups of 16 bytes, so that rows need no alignment; the first of a row's may
// begin in the row before it, and nothing outside the tensor is read (qmm_norm_copy.h).
// What bounds it: memory for many rows (8,192 rows of 5,120, bf16 + fp32 to bf16, us: one norm 65.1, 6.4 TB/s,
// 96 % of a copy; a norm of y too 68.6, 6.1 TB/s; and one row of gates 80, 5.2; a row of gates each
// 104, 5.7), the chain load -> sum -> sum for few (8 rows: 2.6 us), registers past 16,384 entries.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"
#include "qmm_norm_copy.h"

namespace qmm {
namespace {

struct NormParams {
  const void* res;
  const void* y;
  void* res_out;
  void* out;
  int64_t ld_res, ld_y, ld_res_out, ld_out, ld_gate;
  const float* weight;
  const float* bias;
  const float* post_weight;
  const float* post_bias;
  const float* gate;
  int64_t M;
  int N;
  int res_dt, y_dt, out_dt;
  int centered;
  float eps, scale, inv_n;
};

constexpr int SHORT = 64;
constexpr int MAX_DEVICES = 64;

// Entries of a thread: vectors of V, a group's threads side by side.  FULL: the group's
// threads have no places past the row.  FRESH: read once.
template <int E, int V, bool FULL, bool FRESH>
__device__ __forceinline__ void load_row(int dt, const char* row, int t, int threads, int n, float (&x)[E]) {
  if (dt == QMM_DT_F32) {
    const char* at = row + t * V * 4;
    const int step = threads * V * 4;
#pragma unroll
    for (int i = 0; i < E / V; ++i, at += step) {
      const bool in = FULL || (i * threads + t) * V < n;
      if constexpr (V == 4) {
        const float4* q = reinterpret_cast<const float4*>(at);
        const float4 v = in ? (FRESH ? __ldcs(q) : *q) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
      } else {
        const float* q = reinterpret_cast<const float*>(at);
        x[i] = in ? (FRESH ? __ldcs(q) : *q) : 0.f;
      }
    }
    return;
  }
  uint32_t w[(E + 1) / 2];
  const char* at = row + t * V * 2;
  const int step = threads * V * 2;
#pragma unroll
  for (int i = 0; i < E / V; ++i, at += step) {
    const bool in = FULL || (i * threads + t) * V < n;
    if constexpr (V == 4) {
      const uint2* q = reinterpret_cast<const uint2*>(at);
      const uint2 v = in ? (FRESH ? __ldcs(q) : *q) : make_uint2(0u, 0u);
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(at);
      const uint32_t v = in ? (FRESH ? __ldcs(q) : *q) : 0;
      w[i / 2] = i & 1 ? w[i / 2] | v << 16 : v;
    }
  }
  if (dt == QMM_DT_BF16) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = unpack16<false>((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]));
  }
}

template <int E, int V, bool FULL>
__device__ __forceinline__ void store_row(int dt, char* row, int t, int threads, int n, const float (&x)[E]) {
  if (dt == QMM_DT_F32) {
    char* at = row + t * V * 4;
    const int step = threads * V * 4;
#pragma unroll
    for (int i = 0; i < E / V; ++i, at += step) {
      if (!FULL && (i * threads + t) * V >= n) continue;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(at) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      else
        *reinterpret_cast<float*>(at) = x[i];
    }
    return;
  }
  uint32_t w[(E + 1) / 2];
  if (dt == QMM_DT_BF16) {
#pragma unroll
    for (int i = 0; i < E; i += 2) w[i / 2] = pack16<true>(x[i], i + 1 < E ? x[i + 1] : 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 2) w[i / 2] = pack16<false>(x[i], i + 1 < E ? x[i + 1] : 0.f);
  }
  char* at = row + t * V * 2;
  const int step = threads * V * 2;
#pragma unroll
  for (int i = 0; i < E / V; ++i, at += step) {
    if (!FULL && (i * threads + t) * V >= n) continue;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(at) = make_uint2(w[2 * i], w[2 * i + 1]);
    else
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
  }
}

__device__ __forceinline__ int size_of(int dt) { return dt == QMM_DT_F32 ? 4 : 2; }
__device__ __forceinline__ char* row_of(const void* base, int64_t m, int64_t ld, int dt) {
  return const_cast<char*>(static_cast<const char*>(base)) + m * ld * size_of(dt);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// x <- norm(x) w + b; entries past the row stay zero.
template <int E, int V, bool FULL, typename S>
__device__ __forceinline__ void normed(const NormParams& p, float (&x)[E], const float* w, const float* b, int t, int threads,
                                       S sum_all) {
  if (p.centered) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += x[i];
    const float mean = sum_all(s) * p.inv_n;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (FULL || ((i / V) * threads + t) * V + i % V < p.N) x[i] -= mean;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s = fmaf(x[i], x[i], s);
  float wv[E];
  load_row<E, V, FULL, false>(QMM_DT_F32, reinterpret_cast<const char*>(w), t, threads, p.N, wv);
  const float f = rsqrtf(fmaf(sum_all(s), p.inv_n, p.eps));
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = x[i] * f * wv[i];
  if (b) {
    load_row<E, V, FULL, false>(QMM_DT_F32, reinterpret_cast<const char*>(b), t, threads, p.N, wv);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] += wv[i];
  }
}

// One row, from where y, the residual and the gate lie.
template <int E, int V, bool FULL, bool FRESH, typename S>
__device__ __forceinline__ void one_row(const NormParams& p, int64_t m, const char* y, const char* res, const char* gate, int t,
                                        int threads, S sum_all) {
  float r[E];
  load_row<E, V, FULL, FRESH>(p.res_dt, res, t, threads, p.N, r);
  if (p.y) {
    float z[E];
    load_row<E, V, FULL, FRESH>(p.y_dt, y, t, threads, p.N, z);
    if (p.post_weight) normed<E, V, FULL>(p, z, p.post_weight, p.post_bias, t, threads, sum_all);
    if (p.gate) {
      float g[E];
      load_row<E, V, FULL, false>(QMM_DT_F32, gate, t, threads, p.N, g);
#pragma unroll
      for (int i = 0; i < E; ++i) z[i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = fmaf(p.scale, z[i], r[i]);
    store_row<E, V, FULL>(p.res_dt, row_of(p.res_out, m, p.ld_res_out, p.res_dt), t, threads, p.N, r);
  }
  if (p.out) {
    normed<E, V, FULL>(p, r, p.weight, p.bias, t, threads, sum_all);
    store_row<E, V, FULL>(p.out_dt, row_of(p.out, m, p.ld_out, p.out_dt), t, threads, p.N, r);
  }
}

// Short rows: a warp each.  (Against CTAs of a warp, us: 20,000 rows of 7 6.6 : 10.3, of 64 8.3 : 8.6, of 128
// 9.8 : 8.3; with 16 entries a lane, of 384 21.5 : 17.3.)
template <int E, int V>
__global__ void __launch_bounds__(256) norm_short_kernel(const __grid_constant__ NormParams p) {
  const int lane = threadIdx.x & 31;
  for (int64_t m = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); m < p.M; m += (int64_t)gridDim.x * 8)
    one_row<E, V, false, true>(p, m, row_of(p.y, m, p.ld_y, p.y_dt), row_of(p.res, m, p.ld_res, p.res_dt),
                        row_of(p.gate, m, p.ld_gate, QMM_DT_F32), lane, 32, warp_sum);
}

// Longer rows: a CTA each; STAGED: the next one's inputs on their way into shared memory, else
// straight from memory.
template <int E, int V, bool FULL, bool STAGED>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p, int stage_bytes) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float s_sum[2][32];
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5;
  int turn = 0;
  // (sums alternate between two places: a barrier after the writes is enough)
  auto sum_all = [&](float v) {
    v = warp_sum(v);
    if (lane == 0) s_sum[turn][warp] = v;
    __syncthreads();
    v = warp_sum(lane < threads >> 5 ? s_sum[turn][lane] : 0.f);
    turn ^= 1;
    return v;
  };
  if constexpr (!STAGED) {
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x)
      one_row<E, V, FULL, true>(p, m, row_of(p.y, m, p.ld_y, p.y_dt), row_of(p.res, m, p.ld_res, p.res_dt),
                                row_of(p.gate, m, p.ld_gate, QMM_DT_F32), t, threads, sum_all);
    return;
  }
  const int y_bytes = p.N * size_of(p.y_dt), r_bytes = p.N * size_of(p.res_dt);
  const int y_room = p.y ? (y_bytes + 31) & ~15 : 0, r_room = (r_bytes + 31) & ~15;
  const bool gates = p.gate && p.ld_gate;
  // where a row begins behind the boundary that its copy starts from
  auto skew = [](const char* row) { return (int)((uintptr_t)row & 15); };
  auto request = [&](int64_t m, int stage) {
    if (m < p.M) {
      auto copy = [&](int to, const char* row, int bytes) {
        const int s = skew(row);
        row -= s;
        copy_row(
            t, threads, m, s, bytes, [&](int at, int n) { cp_async16(smem_u32(smem) + to + at, row + at, n); },
            [&](int at) { *reinterpret_cast<uint16_t*>(smem + to + at) = *reinterpret_cast<const uint16_t*>(row + at); });
      };
      const int to = stage * stage_bytes;
      if (p.y) copy(to, row_of(p.y, m, p.ld_y, p.y_dt), y_bytes);
      copy(to + y_room, row_of(p.res, m, p.ld_res, p.res_dt), r_bytes);
      if (gates) copy(to + y_room + r_room, row_of(p.gate, m, p.ld_gate, QMM_DT_F32), p.N * 4);
    }
    cp_async_commit();
  };
  int64_t ahead = blockIdx.x;
  request(ahead, 0);
  ahead += gridDim.x;
  int stage = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x, ahead += gridDim.x) {
    // the row has come, and the last one's place is free
    cp_async_wait<0>();
    __syncthreads();
    const char* from = smem + stage * stage_bytes;
    stage ^= 1;
    request(ahead, stage);
    const char* y = from + skew(row_of(p.y, m, p.ld_y, p.y_dt));
    const char* res = from + y_room + skew(row_of(p.res, m, p.ld_res, p.res_dt));
    if (gates)
      one_row<E, V, FULL, false>(p, m, y, res, from + y_room + r_room + skew(row_of(p.gate, m, p.ld_gate, QMM_DT_F32)), t, threads,
                                 sum_all);
    else
      one_row<E, V, FULL, false>(p, m, y, res, reinterpret_cast<const char*>(p.gate), t, threads, sum_all);
  }
}

template <int V>
cudaError_t launch_short(const NormParams& p, int sms, cudaStream_t st) {
  const int64_t need = (p.M + 7) / 8, most = 8ll * sms;
  const unsigned grid = (unsigned)(need < most ? need : most);
  norm_short_kernel<4, V><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

constexpr int SMEM = 220 * 1024;  // of an SM, for stages

template <int E, int V, bool FULL, bool STAGED>
cudaError_t launch_kernel(const NormParams& p, int dev, unsigned grid, int threads, int stage, cudaStream_t st) {
  if (STAGED) {
    static std::atomic<bool> set[MAX_DEVICES];  // once for a device
    if (dev >= MAX_DEVICES || !set[dev].load(std::memory_order_relaxed)) {
      const cudaError_t e = cudaFuncSetAttribute(norm_kernel<E, V, FULL, STAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
      if (e != cudaSuccess) return e;
      if (dev < MAX_DEVICES) set[dev].store(true, std::memory_order_relaxed);
    }
  }
  norm_kernel<E, V, FULL, STAGED><<<grid, threads, STAGED ? 2 * stage : 0, st>>>(p, stage);
  return cudaGetLastError();
}

template <int E, int V>
cudaError_t launch_long(const NormParams& p, int dev, int sms, cudaStream_t st) {
  const int threads = ((p.N + E - 1) / E + 31) / 32 * 32;
  const int ys = p.y_dt == QMM_DT_F32 ? 4 : 2, rs = p.res_dt == QMM_DT_F32 ? 4 : 2;
  const int stage = (p.y ? (p.N * ys + 31) & ~15 : 0) + ((p.N * rs + 31) & ~15) + (p.gate && p.ld_gate ? (p.N * 4 + 31) & ~15 : 0);
  // CTAs that an SM's registers allow (64 a thread), with two stages of shared memory each; more
  // stages leave less for the weights in L1 (8,192 rows of 1,024: 17.6 us with four, 15.9 with two).
  // (Straight from memory 8,192 rows of 5,120 take 77.7 us instead of 68.8, 8,000 of 2,048 35.4
  // instead of 31.1, 2,000 of 16,000 76.6 instead of 70.6.)
  int ctas = 1024 / threads;
  while (ctas > 1 && SMEM / ctas < 2 * stage + 1024) --ctas;
  const int64_t most = (int64_t)ctas * sms;
  // a row alone has no next one to wait for
  const bool staged = SMEM / ctas >= 2 * stage + 1024 && p.M > most;
  const unsigned grid = (unsigned)(p.M < most ? p.M : most);
  const bool full = V == 4 && p.N == threads * E;
  if (staged)
    return full ? launch_kernel<E, V, V == 4, true>(p, dev, grid, threads, stage, st)
                : launch_kernel<E, V, false, true>(p, dev, grid, threads, stage, st);
  return full ? launch_kernel<E, V, V == 4, false>(p, dev, grid, threads, 0, st)
              : launch_kernel<E, V, false, false>(p, dev, grid, threads, 0, st);
}

template <int V>
cudaError_t launch(const NormParams& p, int dev, int sms, cudaStream_t st) {
  if (p.N <= SHORT) return launch_short<V>(p, sms, st);
  // By N alone, so that a row's sums do not depend on how many others there are.  Few rows are
  // done sooner with few entries a thread, many rows want few threads for a sum.  us, of bf16 + fp32
  // to bf16, 4 : 8 entries: 20,000 rows of 128 8.3 : 9.6, of 256 14.6 : 10.8, of 512 26.1 : 18.9; 8 : 16 entries:
  // 8 rows of 777 2.7 : 3.6, 20,000 of 777 47 : 39, of 1,024 34.0 : 34.4, of 1,500 51.7 : 52.3, of 2,048
  // 66.3 : 65.0; 16 : 32 entries, 2,000 rows of 16,000: 69 : 128, for registers.  (Many rows of 513 to
  // 1,023 entries off four would be done sooner with 16, few rows and those on four would not.)
  if (p.N <= 128) return launch_long<4, V>(p, dev, sms, st);
  if (p.N <= 1024) return launch_long<8, V>(p, dev, sms, st);
  return p.N <= 16384 ? launch_long<16, V>(p, dev, sms, st) : launch_long<32, V>(p, dev, sms, st);
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" int qmm_residual_norm(const qmm_norm_args* a, void* stream) {
  if (!a || a->struct_size != sizeof(qmm_norm_args)) return QMM_ERR_INVALID_ARG;
  if (a->res_dtype > QMM_DT_F32 || a->y_dtype > QMM_DT_F32 || a->out_dtype > QMM_DT_F32 || (a->flags & ~QMM_NORM_CENTERED))
    return QMM_ERR_INVALID_ARG;
  if (!a->residual || (!a->y && !a->out) || (a->y && !a->residual_out) || (a->out && !a->weight)) return QMM_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || !isfinite(a->eps) || !isfinite(a->scale)) return QMM_ERR_INVALID_ARG;
  if (a->M < 1 || a->M > INT32_MAX || a->N < 1 || a->N > QMM_NORM_MAX_N) return QMM_ERR_SHAPE;
  const int rs = a->res_dtype == QMM_DT_F32 ? 4 : 2, ys = a->y_dtype == QMM_DT_F32 ? 4 : 2,
            os = a->out_dtype == QMM_DT_F32 ? 4 : 2;
  const uintptr_t res = (uintptr_t)a->residual | (a->y ? (uintptr_t)a->residual_out : 0), y = (uintptr_t)a->y,
                  out = (uintptr_t)a->out,
                  f32 = (uintptr_t)a->weight | (uintptr_t)a->bias | (uintptr_t)a->post_weight | (uintptr_t)a->post_bias |
                        (uintptr_t)a->gate;
  if ((res & (rs - 1)) || (y & (ys - 1)) || (out & (os - 1)) || (f32 & 3)) return QMM_ERR_ALIGN;
  if (a->M > 1 && (a->ld_residual < a->N || (a->y && (a->ld_y < a->N || a->ld_residual_out < a->N)) ||
                   (a->out && a->ld_out < a->N) || (a->gate && a->ld_gate && a->ld_gate < a->N)))
    return QMM_ERR_ALIGN;
  // onto an input: every element is read by the thread that writes it, if it stays where it is
  auto moves = [&](const void* to, int64_t ld, int size, const void* from, int64_t ld_from, int size_from) {
    return to && to == from && (size != size_from || (a->M > 1 && ld != ld_from));
  };
  auto onto = [&](const void* to, int64_t ld, int size) {
    return moves(to, ld, size, a->residual, a->ld_residual, rs) || moves(to, ld, size, a->y, a->ld_y, ys) ||
           (a->y && moves(to, ld, size, a->gate, a->ld_gate, 4));
  };
  if ((a->y && a->residual_out == a->out) || (a->y && onto(a->residual_out, a->ld_residual_out, rs)) || onto(a->out, a->ld_out, os))
    return QMM_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  const int rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  // weights and biases are read for every row: no row of an output may touch them
  auto touches = [&](const void* to, int64_t ld, int size, const float* vec) {
    if (!to || !vec) return false;
    const int64_t row = a->N * size, step = a->M > 1 ? ld * size : row, len = a->N * 4;
    const int64_t d = (int64_t)((uintptr_t)vec - (uintptr_t)to);  // of the vector behind the first row's start
    if (d < 0) return d + len > 0;
    const int64_t m = d / step;  // the last row that begins at or before the vector
    return (m < a->M && d - m * step < row) || (m + 1 < a->M && d + len > (m + 1) * step);
  };
  auto over = [&](const float* vec) {
    return (a->y && touches(a->residual_out, a->ld_residual_out, rs, vec)) || touches(a->out, a->ld_out, os, vec);
  };
  if ((a->out && (over(a->weight) || over(a->bias))) || (a->y && (over(a->post_weight) || over(a->post_bias))))
    return QMM_ERR_INVALID_ARG;
  NormParams p;
  p.res = a->residual, p.y = a->y, p.res_out = a->residual_out, p.out = a->out;
  const bool many = a->M > 1;  // the stride of a single row is not followed
  p.ld_res = many ? a->ld_residual : 0;
  p.ld_y = many && a->y ? a->ld_y : 0;
  p.ld_res_out = many && a->y ? a->ld_residual_out : 0;
  p.ld_out = many && a->out ? a->ld_out : 0;
  p.ld_gate = many && a->gate ? a->ld_gate : 0;
  p.weight = a->weight, p.bias = a->bias;
  p.post_weight = a->post_weight, p.post_bias = a->post_bias;
  p.gate = a->y ? a->gate : nullptr;  // (rows ahead are copied with their gates)
  p.M = a->M;
  p.N = (int)a->N;
  p.res_dt = a->res_dtype, p.y_dt = a->y_dtype, p.out_dt = a->out_dtype;
  p.centered = a->flags & QMM_NORM_CENTERED ? 1 : 0;
  p.eps = a->eps, p.scale = a->scale;
  p.inv_n = 1.f / (float)p.N;
  // vectors of four where every one of them lies on its boundary
  const bool wide = !((p.N | p.ld_res | p.ld_y | p.ld_res_out | p.ld_out | p.ld_gate) & 3) && !(res & (4 * rs - 1)) &&
                    !(y & (4 * ys - 1)) && !(out & (4 * os - 1)) && !(f32 & 15);
  const cudaError_t e = wide ? launch<4>(p, dev, sms, (cudaStream_t)stream) : launch<1>(p, dev, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}
