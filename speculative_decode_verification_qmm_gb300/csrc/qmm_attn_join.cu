// qmm_attn_join.cu -- adds up the partial results of attention items that were
// cut between CTAs (qmm_attn.cuh).
//
//   m = max m_c,  l = sum l_c 2^(m_c - m),  O = sum O_c 2^(m_c - m),  out = O / l
// over the item's CTAs c in order.  The partials are read from L2; what bounds
// the kernel is latency, so the work is spread over the GPU (RU rows of one
// item per warp), loads of several parts and rows are in flight at a time, and
// everything that does not depend on the partials is done before the wait for
// the kernel that writes them (programmatic dependent launch).  As a tail of the
// attention kernels' last CTA of an item the same sums took up to 30 us (64
// items of 256 rows, 4 parts each), because one SM had to read them all.
#include <cuda_runtime.h>

#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {

namespace {

constexpr int WARPS = 4;
constexpr int RU = 2;  // rows of a lane

template <bool BF16, int D>
__global__ void __launch_bounds__(WARPS * 32) attn_join_kernel(const __grid_constant__ AttnParams p, int tk, int rows,
                                                               int chunks) {
  constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes of a row, rows of a warp at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
  AttnCursor cur{};
  cur.b = item / (p.Hkv * p.RT);
  cur.h = item / p.RT % p.Hkv;
  cur.rt = item % p.RT;
  attn_sizes(p, cur.b, cur.L, cur.n);
  int nt = (cur.L + cur.n + tk - 1) / tk;
  nt = nt < 1 ? 1 : nt;
  int64_t before, all;
  attn_count(p, tk, lane, cur.b, before, all);
  const int64_t W = all * p.Hkv * p.RT;
  const int G = W < p.grid ? (int)W : p.grid;
  const int64_t u = before * p.Hkv * p.RT + (int64_t)(cur.h * p.RT + cur.rt) * nt;
  const int c0 = attn_owner(u, W, G), c1 = attn_owner(u + nt - 1, W, G);
  const int part = rows * (D + 2);
  const int r0 = (chunk * WARPS + warp) * RPW * RU + lane / LPR;
  const int left = p.R - cur.rt * rows < rows ? p.R - cur.rt * rows : rows;
  const int sub = lane % LPR, c4 = sub * 4;
  pdl_wait();  // every CTA: the call has not ended before the attention kernel has
  if (c0 == c1 || r0 - lane / LPR >= left) return;

  float4 acc[RU];
  float mn[RU], lt[RU];
#pragma unroll
  for (int k = 0; k < RU; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f), mn[k] = -INFINITY, lt[k] = 0.f;
  for (int cb = c0; cb <= c1; cb += LPR) {
    // each lane of a row takes one part's statistics
    const int mine = cb + sub;
    float m[RU], l[RU], w[RU];
#pragma unroll
    for (int k = 0; k < RU; ++k) {
      m[k] = -INFINITY, l[k] = 0.f;
      if (mine <= c1) {
        const float* pp = p.ws + ((int64_t)mine * 2 + (mine == c0)) * part + rows * D + r0 + k * RPW;
        m[k] = __ldcg(pp);
        l[k] = __ldcg(pp + rows);
      }
    }
#pragma unroll
    for (int k = 0; k < RU; ++k) {
      float x = m[k];
#pragma unroll
      for (int d = LPR / 2; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
      x = fmaxf(x, mn[k]);
      const float old = attn_weight(mn[k], lt[k], x);
      w[k] = attn_weight(m[k], l[k], x);
      float sum = w[k] * l[k];
#pragma unroll
      for (int d = LPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      lt[k] = lt[k] * old + sum;
      acc[k].x *= old, acc[k].y *= old, acc[k].z *= old, acc[k].w *= old;
      mn[k] = x;
    }
    const int n = c1 - cb + 1 < LPR ? c1 - cb + 1 : LPR;
    constexpr int U = 4;
    for (int i = 0; i < n; i += U) {
      float4 v[U][RU];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < RU; ++k) {
          v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          const int c = cb + i + j;
          if (c <= c1 && i + j < n)
            v[j][k] = __ldcg(reinterpret_cast<const float4*>(p.ws + ((int64_t)c * 2 + (c == c0)) * part +
                                                             (r0 + k * RPW) * D + c4));
        }
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < RU; ++k) {
          const float x = __shfl_sync(0xFFFFFFFFu, w[k], i + j < n ? i + j : 0, LPR);
          if (i + j < n)
            acc[k].x += x * v[j][k].x, acc[k].y += x * v[j][k].y, acc[k].z += x * v[j][k].z, acc[k].w += x * v[j][k].w;
        }
    }
  }
#pragma unroll
  for (int k = 0; k < RU; ++k)
    if (r0 + k * RPW < left) attn_store4<BF16>(p, cur, cur.rt * rows + r0 + k * RPW, c4, acc[k], mn[k], lt[k]);
}

template <bool BF16, int D>
cudaError_t launch(const AttnParams& p, int tk, int rows, cudaStream_t st) {
  constexpr int PER = WARPS * (128 / D) * RU;
  const int chunks = ((p.R < rows ? p.R : rows) + PER - 1) / PER;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * p.RT * chunks));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<BF16, D>, p, tk, rows, chunks);
}

}  // namespace

cudaError_t launch_attn_join(const AttnParams& p, bool bf16, int D, int tk, int rows, cudaStream_t st) {
  if (D == 128) return bf16 ? launch<true, 128>(p, tk, rows, st) : launch<false, 128>(p, tk, rows, st);
  return bf16 ? launch<true, 64>(p, tk, rows, st) : launch<false, 64>(p, tk, rows, st);
}

}  // namespace qmm
