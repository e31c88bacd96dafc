// qmm_attn_join.cu -- adds up the partial results of attention items that were
// cut between CTAs (qmm_attn.cuh).
//
//   m = max m_c,  l = sum l_c 2^(m_c - m),  O = sum O_c 2^(m_c - m),  out = O / l
// over the item's CTAs c.  The partials are read from L2; what bounds the kernel
// is latency, so a CTA takes four rows (eight at head size 64) at a time, its four
// warps every fourth part of them, and all of a warp's loads of two parts are in
// flight at a time; the warps' sums are added in order through shared memory.
// An item of four parts or fewer and many rows gives each warp rows of its own (4 x
// 16,384 rows, 512 rows a head: 7 us less).
// Where there are more rows than eight CTAs an SM would take, a CTA goes on to
// further ones: finding its item costs as much as four of them (four CTAs an SM:
// 4 us more, 32: 5 us more).  What it adds to the attention kernel: 5 to 10 us where all
// items are cut, 2 where none is.
// Most of more items than that are not cut.  The CTAs are then for the workers:
// each reads what its worker left (AttnParams::cuts) and joins the item that goes
// on behind the worker's range, if one began in it.
// Items of the prompt attention (qmm_prompt.cu) are joined by cuts always; there a cut
// holds the item's first row among the packed ones, its head and its number of rows.  A
// few long items can be all that there is: the CTAs share out the cuts that begin an item, as many
// to each (64 rows of 32 heads of 64 behind 20,000: 38 us with CTAs for every worker, so 24;
// 1,024 rows, 12 heads of 128: 23 and 21).
// Everything that does not depend on the partials is done before the wait for
// the kernel that writes them (programmatic dependent launch).  As a tail of the
// attention kernels' last CTA of an item the same sums took up to 30 us (64
// items of 256 rows, 4 parts each), because one SM had to read them all.
#include <cuda_runtime.h>

#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {

namespace {

constexpr int WARPS = 4;
constexpr int RU = 4;  // rows of a lane
constexpr int U = 2;   // parts in flight
constexpr int CTAS_PER_SM = 8;
constexpr int GRID_MAX = ATTN_PROMPT_GRID_MAX;
enum { ITEMS, CUTS_OF_TREES, CUTS_OF_PROMPTS };

template <bool BF16, int D, int MODE>
__global__ void __launch_bounds__(WARPS * 32, D == 128 ? 7 : 5) attn_join_kernel(const __grid_constant__ AttnParams p, int tk, int rows,
                                                               int chunks) {
  constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes of a row, rows of a warp's load
  constexpr int RPC = RPW * RU;               // rows of the CTA
  constexpr bool CUTS = MODE != ITEMS, PROMPT = MODE == CUTS_OF_PROMPTS;
  __shared__ float4 s_acc[WARPS][RPC][LPR];
  __shared__ float s_m[WARPS][RPC], s_l[WARPS][RPC];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int unit = blockIdx.x / chunks, chunk = blockIdx.x - unit * chunks;
  AttnCursor cur{};
  int c0 = unit, c1 = unit;
  if constexpr (!CUTS) {
    cur.b = unit / (p.Hkv * p.RT);
    cur.h = unit / p.RT % p.Hkv;
    cur.rt = unit % p.RT;
    attn_sizes(p, cur.b, cur.L, cur.n);
    int nt = (cur.L + cur.n + tk - 1) / tk;
    nt = nt < 1 ? 1 : nt;
    int64_t before, all;
    attn_count(p, tk, lane, cur.b, before, all);
    const int64_t W = all * p.Hkv * p.RT;
    const int G = W < p.grid ? (int)W : p.grid;
    const int64_t u = before * p.Hkv * p.RT + (int64_t)(cur.h * p.RT + cur.rt) * nt;
    c0 = attn_owner(u, W, G);
    c1 = attn_owner(u + nt - 1, W, G);
  }
  pdl_wait();  // every CTA: the call has not ended before the attention kernel has
  if constexpr (PROMPT) {
    // The CTAs share out the cuts that begin an item, as one warp finds them.  (By all four, 1.5 us more.)
    __shared__ int s_item[6];
    if (warp == 0) {
      int4 cut[GRID_MAX / 32];
      unsigned begins[GRID_MAX / 32];
      int n = 0;
#pragma unroll
      for (int k = 0; k < GRID_MAX / 32; ++k)
        cut[k] = k * 32 + lane + 1 < p.grid ? __ldcg(p.cuts + k * 32 + lane) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < GRID_MAX / 32; ++k) {
        begins[k] = __ballot_sync(0xFFFFFFFFu, cut[k].w == 1);
        n += __popc(begins[k]);
      }
      chunk = n ? blockIdx.x / n : 0;
      unit = n ? blockIdx.x - chunk * n : 0;
      c0 = c1 = -1;
#pragma unroll
      for (int k = 0; k < GRID_MAX / 32; ++k) {
        const bool here = cut[k].w == 1 && __popc(begins[k] & ((1u << lane) - 1)) == unit;
        if (here) s_item[3] = cut[k].x, s_item[4] = cut[k].y, s_item[5] = cut[k].z;
        const unsigned at = __ballot_sync(0xFFFFFFFFu, here);
        if (at) c0 = k * 32 + __ffs(at) - 1;
        unit -= __popc(begins[k]);
      }
#pragma unroll
      for (int k = 0; k < GRID_MAX / 32; ++k) {
        // the first worker from the next one on whose last unit is not of this item
        const unsigned end = __ballot_sync(0xFFFFFFFFu, k * 32 + lane > c0 && cut[k].w != 2);
        if (end && c1 < 0) c1 = k * 32 + __ffs(end) - 1;
      }
      if (lane == 0) s_item[0] = n, s_item[1] = c0, s_item[2] = c1;
    }
    __syncthreads();
    const int n = s_item[0];
    if (n == 0) return;
    chunks = gridDim.x / n;  // (n < grid <= gridDim.x)
    chunk = blockIdx.x / n;
    if (chunk >= chunks) return;
    c0 = s_item[1], c1 = s_item[2];
    cur.b = s_item[3], cur.h = s_item[4], cur.rt = s_item[5];
  } else if constexpr (CUTS) {
    const int4 cut = __ldcg(p.cuts + c0);
    if (cut.w == 1) {
      // the first worker from the next one on whose last unit is not of this item,
      // 32 at a time: one after the other, 1,300 sequences of 16 rows and one
      // of 131,072 with one head took 120 us, and take 91
      for (c1 = c0 + 1;; c1 += 32) {
        const bool on = c1 + lane + 1 < p.grid && __ldcg(&p.cuts[c1 + lane].w) == 2;
        const unsigned end = __ballot_sync(0xFFFFFFFFu, !on);
        if (end) {
          c1 += __ffs(end) - 1;
          break;
        }
      }
    }
    cur.b = cut.x, cur.h = cut.y, cur.rt = cut.z;
  }
  if (c0 == c1) return;
  const int part = rows * (D + 2);
  int left, first_row;  // the item's rows, and the first one's place among the head's
  if constexpr (PROMPT) {
    first_row = cur.b * p.g, left = cur.rt;
    cur.b = 0, cur.n = INT32_MAX;
  } else {
    if constexpr (CUTS) attn_sizes(p, cur.b, cur.L, cur.n);
    first_row = cur.rt * rows;
    left = p.R - first_row < rows ? p.R - first_row : rows;
  }
  const int sub = lane % LPR, row = lane / LPR;

  // a warp joins its rows alone
  const bool alone = c1 - c0 < 4 && (PROMPT ? chunks * RPC < left : CUTS || left >= 128);
  const int from = alone ? c0 : c0 + warp, step = alone ? 1 : WARPS;
  const int first = alone ? (chunk * WARPS + warp) * RPC : chunk * RPC;
  const int hop = chunks * (alone ? WARPS * RPC : RPC);
  for (int r0 = first; r0 < left; r0 += hop) {
    float4 acc[RU];
    float mn[RU], lt[RU];
#pragma unroll
    for (int k = 0; k < RU; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f), mn[k] = -INFINITY, lt[k] = 0.f;
    for (int c = from; c <= c1; c += step * U) {
      float4 v[U][RU];
      float m[U][RU], l[U][RU];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int cc = c + j * step;
        const float* pp = p.ws + ((int64_t)cc * 2 + (cc == c0)) * part;
#pragma unroll
        for (int k = 0; k < RU; ++k) {
          const int r = r0 + k * RPW + row;
          const bool have = cc <= c1;  // (rows past the item's are in the workspace too)
          m[j][k] = have ? __ldcg(pp + rows * D + r) : -INFINITY;
          l[j][k] = have ? __ldcg(pp + rows * D + rows + r) : 0.f;
          v[j][k] = have ? __ldcg(reinterpret_cast<const float4*>(pp + r * D) + sub) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < RU; ++k) {
          const float x = fmaxf(mn[k], m[j][k]);
          const float a = attn_weight(mn[k], lt[k], x), w = attn_weight(m[j][k], l[j][k], x);
          lt[k] = lt[k] * a + l[j][k] * w;
          acc[k].x = acc[k].x * a + v[j][k].x * w;
          acc[k].y = acc[k].y * a + v[j][k].y * w;
          acc[k].z = acc[k].z * a + v[j][k].z * w;
          acc[k].w = acc[k].w * a + v[j][k].w * w;
          mn[k] = x;
        }
    }
    if (alone) {
#pragma unroll
      for (int k = 0; k < RU; ++k) {
        const int r = r0 + k * RPW + row;
        if (r < left) attn_store4<BF16>(p, cur, first_row + r, sub * 4, acc[k], mn[k], lt[k]);
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < RU; ++k) {
      s_acc[warp][k * RPW + row][sub] = acc[k];
      if (sub == 0) {
        s_m[warp][k * RPW + row] = mn[k];
        s_l[warp][k * RPW + row] = lt[k];
      }
    }
    __syncthreads();
    // one thread a float4 of a row
    const int rr = threadIdx.x / LPR;
    static_assert(RPC * LPR == WARPS * 32, "a thread for each float4");
    if (r0 + rr < left) {
      float mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, s_m[w][rr]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float x = attn_weight(s_m[w][rr], s_l[w][rr], mx);
        const float4 v = s_acc[w][rr][sub];
        l += s_l[w][rr] * x;
        a.x += v.x * x, a.y += v.y * x, a.z += v.z * x, a.w += v.w * x;
      }
      attn_store4<BF16>(p, cur, first_row + r0 + rr, sub * 4, a, mx, l);
    }
    __syncthreads();
  }
}

template <bool BF16, int D, int MODE>
cudaError_t launch(const AttnParams& p, int tk, int rows, int ctas, cudaStream_t st) {
  constexpr bool CUTS = MODE != ITEMS;
  constexpr int PER = 128 / D * RU * (CUTS ? WARPS : 1);
  const int64_t units = CUTS ? p.grid - 1 : (int64_t)p.B * p.Hkv * p.RT;
  int chunks = ((p.R < rows ? p.R : rows) + PER - 1) / PER;
  const int64_t most = (ctas + units - 1) / units;
  if (chunks > most) chunks = (int)most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(MODE == CUTS_OF_PROMPTS ? ctas : units * chunks));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<BF16, D, MODE>, p, tk, rows, chunks);
}

template <bool BF16, int D>
cudaError_t launch_one(const AttnParams& p, int tk, int rows, int sms, cudaStream_t st) {
  // Measured, CTAs by cuts against by items, in us with the attention kernel:
  // 2,560 items (128 sequences of up to 120 / 600 / 4,000 rows, head size 64): 36 :
  // 43, 68 : 78, 296 : 299; 5,120 (head size 128, up to 120 / 300 / 800): 87 : 103, 128
  // : 143, 212 : 222; 320 (16 sequences, up to 120 / 600 / 4,000): 18 : 17, 30 : 29,
  // 91 : 89; 384 (48 sequences, 8 heads): 13.6 : 13.1, 28 : 27, 90 : 88.
  const int ctas = CTAS_PER_SM * sms;
  const bool cuts = (int64_t)p.B * p.Hkv * p.RT > ctas;
  return cuts ? launch<BF16, D, CUTS_OF_TREES>(p, tk, rows, ctas, st) : launch<BF16, D, ITEMS>(p, tk, rows, ctas, st);
}

template <bool BF16, int D>
cudaError_t launch_prompts(const AttnParams& p, int rows, int sms, cudaStream_t st) {
  return p.grid > 1 ? launch<BF16, D, CUTS_OF_PROMPTS>(p, 0, rows, (D == 128 ? 7 : CTAS_PER_SM) * sms, st) : cudaSuccess;
}

}  // namespace

cudaError_t launch_prompt_join(const AttnParams& p, bool bf16, int D, int rows, int sms, cudaStream_t st) {
  if (D == 128) return bf16 ? launch_prompts<true, 128>(p, rows, sms, st) : launch_prompts<false, 128>(p, rows, sms, st);
  return bf16 ? launch_prompts<true, 64>(p, rows, sms, st) : launch_prompts<false, 64>(p, rows, sms, st);
}

cudaError_t launch_attn_join(const AttnParams& p, bool bf16, int D, int tk, int rows, int sms, cudaStream_t st) {
  if (D == 128) return bf16 ? launch_one<true, 128>(p, tk, rows, sms, st) : launch_one<false, 128>(p, tk, rows, sms, st);
  return bf16 ? launch_one<true, 64>(p, tk, rows, sms, st) : launch_one<false, 64>(p, tk, rows, sms, st);
}

}  // namespace qmm
