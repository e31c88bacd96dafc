// qmm_norm.cu -- residual sums with the norms before and after a block
// (qmm_residual_norm in include/qmm.h).
//
// Mathematics.  z = y or norm(y) w_p + b_p;  r' = r + s g z;  out = norm(r') w + b,
// norm(x) = x rsqrt(mean x^2 + eps), or of x - mean x: the mean first, then the mean
// square of the differences, which does not cancel.
//
// A group of threads (a warp for short rows, else the CTA) holds a whole row in
// registers, E entries a thread, so that every input is read once and r' is
// normalised unrounded.
// What bounds it: memory for many rows, the chain load -> sum -> load for few.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"

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

// Entries of a thread: vectors of V, a group's threads side by side.
template <int E, int V>
__device__ __forceinline__ void load_row(int dt, const void* base, int64_t at, int t, int threads, int n, float (&x)[E]) {
  if (dt == QMM_DT_F32) {
    const float* p = static_cast<const float*>(base) + at;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int k = (i * threads + t) * V;
      if constexpr (V == 4) {
        const float4 v = k < n ? *reinterpret_cast<const float4*>(p + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
      } else {
        x[i] = k < n ? p[k] : 0.f;
      }
    }
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  const bool bf = dt == QMM_DT_BF16;
  auto wide = [&](uint32_t v) { return bf ? unpack16<true>((uint16_t)v) : unpack16<false>((uint16_t)v); };
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int k = (i * threads + t) * V;
    if constexpr (V == 4) {
      const uint2 v = k < n ? *reinterpret_cast<const uint2*>(p + k) : make_uint2(0u, 0u);
      x[4 * i] = wide(v.x), x[4 * i + 1] = wide(v.x >> 16), x[4 * i + 2] = wide(v.y), x[4 * i + 3] = wide(v.y >> 16);
    } else {
      x[i] = k < n ? wide(p[k]) : 0.f;
    }
  }
}

template <int E, int V>
__device__ __forceinline__ void store_row(int dt, void* base, int64_t at, int t, int threads, int n, const float (&x)[E]) {
  if (dt == QMM_DT_F32) {
    float* p = static_cast<float*>(base) + at;
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const int k = (i * threads + t) * V;
      if (k >= n) continue;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(p + k) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      else
        p[k] = x[i];
    }
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  const bool bf = dt == QMM_DT_BF16;
  auto pack = [&](float a, float b) { return bf ? pack16<true>(a, b) : pack16<false>(a, b); };
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    const int k = (i * threads + t) * V;
    if (k >= n) continue;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p + k) = make_uint2(pack(x[4 * i], x[4 * i + 1]), pack(x[4 * i + 2], x[4 * i + 3]));
    else
      p[k] = (uint16_t)pack(x[i], 0.f);
  }
}

template <bool WARP, int E, int V>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = WARP ? 32 : blockDim.x, t = WARP ? lane : threadIdx.x;
  const int64_t rows = WARP ? (int64_t)gridDim.x * (blockDim.x / 32) : gridDim.x;
  auto sum_all = [&](float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (!WARP) {
      __syncthreads();  // the sums before were read
      if (lane == 0) s_sum[warp] = v;
      __syncthreads();
      v = lane < (int)(blockDim.x / 32) ? s_sum[lane] : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    }
    return v;
  };
  // x <- norm(x) w + b; entries past the row stay zero
  auto normed = [&](float (&x)[E], const float* w, const float* b) {
    if (p.centered) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) s += x[i];
      const float mean = sum_all(s) * p.inv_n;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (((i / V) * threads + t) * V + i % V < p.N) x[i] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(x[i], x[i], s);
    const float f = rsqrtf(fmaf(sum_all(s), p.inv_n, p.eps));
    float wv[E];
    load_row<E, V>(QMM_DT_F32, w, 0, t, threads, p.N, wv);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = x[i] * f * wv[i];
    if (b) {
      load_row<E, V>(QMM_DT_F32, b, 0, t, threads, p.N, wv);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] += wv[i];
    }
  };
  for (int64_t m = WARP ? (int64_t)blockIdx.x * (blockDim.x / 32) + warp : blockIdx.x; m < p.M; m += rows) {
    float r[E];
    load_row<E, V>(p.res_dt, p.res, m * p.ld_res, t, threads, p.N, r);
    if (p.y) {
      float z[E];
      load_row<E, V>(p.y_dt, p.y, m * p.ld_y, t, threads, p.N, z);
      if (p.post_weight) normed(z, p.post_weight, p.post_bias);
      if (p.gate) {
        float g[E];
        load_row<E, V>(QMM_DT_F32, p.gate, m * p.ld_gate, t, threads, p.N, g);
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) r[i] = fmaf(p.scale, z[i], r[i]);
      store_row<E, V>(p.res_dt, p.res_out, m * p.ld_res_out, t, threads, p.N, r);
    }
    if (p.out) {
      normed(r, p.weight, p.bias);
      store_row<E, V>(p.out_dt, p.out, m * p.ld_out, t, threads, p.N, r);
    }
  }
}

template <int V>
cudaError_t launch(const NormParams& p, int sms, cudaStream_t st) {
  if (p.N <= 1024) {
    const int64_t need = (p.M + 7) / 8, most = 8ll * sms;
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (p.N <= 128)
      norm_kernel<true, 4, V><<<grid, 256, 0, st>>>(p);
    else if (p.N <= 512)
      norm_kernel<true, 16, V><<<grid, 256, 0, st>>>(p);
    else
      norm_kernel<true, 32, V><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  const int E = p.N <= 8192 ? 8 : (p.N <= 16384 ? 16 : 32);
  const int threads = ((p.N + E - 1) / E + 31) / 32 * 32;
  const int64_t most = 2048ll / threads * sms * (E == 8 ? 1 : 1);
  const unsigned grid = (unsigned)(p.M < most ? p.M : most);
  if (E == 8)
    norm_kernel<false, 8, V><<<grid, threads, 0, st>>>(p);
  else if (E == 16)
    norm_kernel<false, 16, V><<<grid, threads, 0, st>>>(p);
  else
    norm_kernel<false, 32, V><<<grid, threads, 0, st>>>(p);
  return cudaGetLastError();
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
  int dev = 0, sms = 0;
  const int rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  NormParams p;
  p.res = a->residual, p.y = a->y, p.res_out = a->residual_out, p.out = a->out;
  const bool many = a->M > 1;  // the stride of a single row is not followed
  p.ld_res = many ? a->ld_residual : 0;
  p.ld_y = many && a->y ? a->ld_y : 0;
  p.ld_res_out = many && a->y ? a->ld_residual_out : 0;
  p.ld_out = many && a->out ? a->ld_out : 0;
  p.ld_gate = many && a->gate ? a->ld_gate : 0;
  p.weight = a->weight, p.bias = a->bias;
  p.post_weight = a->post_weight, p.post_bias = a->post_bias, p.gate = a->gate;
  p.M = a->M;
  p.N = (int)a->N;
  p.res_dt = a->res_dtype, p.y_dt = a->y_dtype, p.out_dt = a->out_dtype;
  p.centered = a->flags & QMM_NORM_CENTERED ? 1 : 0;
  p.eps = a->eps, p.scale = a->scale;
  p.inv_n = 1.f / (float)p.N;
  // vectors of four where every one of them lies on its boundary
  const bool wide = !((p.N | p.ld_res | p.ld_y | p.ld_res_out | p.ld_out | p.ld_gate) & 3) && !(res & (4 * rs - 1)) &&
                    !(y & (4 * ys - 1)) && !(out & (4 * os - 1)) && !(f32 & 15);
  const cudaError_t e = wide ? launch<4>(p, sms, (cudaStream_t)stream) : launch<1>(p, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}
