// qmm_attn.cuh -- what the tree-attention kernels share: launch parameters, the
// division of a batch's work over the grid, and the joining of partial results.
//
// Work.  The rows of one (sequence, key/value head) are the T * g pairs of a
// node and one of the g query heads that read the head: row r = t * g + i.  An
// item is one row tile of one (sequence, head); its units are tiles of
// consecutive cache rows.  All units of the call, ordered (sequence, head, row
// tile, cache tile), are cut into equal contiguous ranges, one per CTA, so that
// ragged batches and single long sequences load the SMs alike and no plan is
// needed from the host, which does not know the lengths.  A CTA's part of an
// item is a segment.  An item that is one segment is written out directly; the
// others leave (O, m, l) partials in the workspace, at most two of a CTA, which
// a second kernel (qmm_attn_join.cu) adds up in CTA order.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm_common.cuh"

namespace qmm {

constexpr int DEV_ERR_INDEX = 16;  // a length, page id or path entry out of range

struct AttnParams {
  const uint16_t* q;
  const uint16_t* kn;
  const uint16_t* vn;
  uint16_t* out;
  int64_t q_sb, q_st, q_sh;
  int64_t k_sb, k_st, k_sh;
  int64_t v_sb, v_st, v_sh;
  int64_t o_sb, o_st, o_sh;
  float* lse;
  uint16_t* k_pool;  // of the layer
  uint16_t* v_pool;
  int64_t page_stride;  // elements of one page: n_kv_heads * page_size * D
  int64_t n_pages;
  const int32_t* table;
  int64_t ld_table;
  int table_width;
  int page_shift;
  const int32_t* lens;
  const int32_t* n_tokens;
  const uint64_t* mask;
  int64_t ld_mask;
  int B, T, Hq, Hkv, g;
  int R;    // rows of an item's head: T * g
  int RT;   // row tiles
  float scale_log2;  // scale * log2(e): the softmax runs in powers of two
  float* ws;         // partials: [worker][2][rows of a tile * (D + 2)]
  int grid;          // workers that share the units: CTAs, or warps that work alone
  int4* cuts;        // [worker]: sequence, head, row tile of its last unit, and attn_cut of it
  int64_t row0;      // first row of the layer in the pools' tensor maps
  int* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                                  uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// 16-byte asynchronous copy global -> shared; `bytes` 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 values as a pair of the 16-bit type (first in the low half).
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float unpack16(uint16_t v) {
  if constexpr (BF16) return __uint_as_float((uint32_t)v << 16);
  return __half2float(__ushort_as_half(v));
}
// Whether any of the eight 16-bit values is an infinity or a NaN: exponent bits all ones.
template <bool BF16>
__device__ __forceinline__ bool any_nonfinite(const uint4& v) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (w[i] & E) == E || ((w[i] >> 16) & E) == E;
  return bad;
}
// The same pair-wise: zero in the place of every non-finite value.
template <bool BF16>
__device__ __forceinline__ uint32_t zero_nonfinite(uint32_t w) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  if ((w & E) == E) w &= 0xFFFF0000u;
  if (((w >> 16) & E) == E) w &= 0x0000FFFFu;
  return w;
}

// The kernels' running maximum m, the base of P = 2^(c s - m), is the row's largest
// c s less this: 0 in bf16, whose range P needs no part of.  In f16 what lies below
// 2^-25 is lost from P V (not from the sum l): with the largest P between 2^7 and,
// as m may lag by 8, 2^15, that is 2^-32 of the largest, or 3e-5 over 131,072 rows
// instead of 4e-3.
template <bool BF16>
constexpr float ATTN_BASE_BELOW = BF16 ? 0.f : 7.f;

// Cached rows L and nodes n of sequence b, brought into the range that the
// page table can hold (what is out of range is reported, not followed).
__device__ __forceinline__ bool attn_sizes(const AttnParams& p, int b, int& L, int& n) {
  const int64_t cap = (int64_t)p.table_width << p.page_shift;
  L = __ldg(p.lens + b);
  n = p.n_tokens ? __ldg(p.n_tokens + b) : p.T;
  bool ok = L >= 0 && n >= 0 && n <= p.T && (int64_t)L + n <= cap;
  if (!ok) {
    L = L < 0 ? 0 : L;
    n = n < 0 ? 0 : (n > p.T ? p.T : n);
    if (L > cap) L = (int)cap;
    if ((int64_t)L + n > cap) n = (int)(cap - L);
  }
  return ok;
}

// A position in the call's units: sequence, head, row tile, cache tile.
struct AttnCursor {
  int b, h, rt, tile, ntiles, L, n;
};

template <int TK>
__device__ __forceinline__ int attn_tiles(int L, int n) {
  const int t = (L + n + TK - 1) / TK;
  return t < 1 ? 1 : t;  // an item without rows still writes its outputs
}

// Cache tiles of the sequences before b, and of all, in every lane of a warp.
__device__ __forceinline__ void attn_count(const AttnParams& p, int tk, int lane, int b, int64_t& before, int64_t& all) {
  before = all = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int nt = 0;
    if (b0 + lane < p.B) {
      int L, n;
      attn_sizes(p, b0 + lane, L, n);
      nt = (L + n + tk - 1) / tk;
      nt = nt < 1 ? 1 : nt;
    }
    all += __reduce_add_sync(0xFFFFFFFFu, nt);
    before += __reduce_add_sync(0xFFFFFFFFu, b0 + lane < b ? nt : 0);
  }
}

// The cursor at the first unit of CTA c's range [u0, u1), for every lane of a
// warp (all lanes call it).
template <int TK>
__device__ __forceinline__ AttnCursor attn_begin(const AttnParams& p, int lane, int c, int64_t& u0, int64_t& u1) {
  const int64_t hr = (int64_t)p.Hkv * p.RT;
  int64_t sum = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int nt = 0;
    if (b0 + lane < p.B) {
      int L, n;
      if (!attn_sizes(p, b0 + lane, L, n) && c == 0) atomicOr(p.status, DEV_ERR_INDEX);
      nt = attn_tiles<TK>(L, n);
    }
    sum += __reduce_add_sync(0xFFFFFFFFu, nt);
  }
  const int64_t W = sum * hr;
  const int G = W < p.grid ? (int)W : p.grid;
  AttnCursor cur{};
  if (c >= G) {
    u0 = u1 = 0;
    return cur;
  }
  u0 = W * c / G;
  u1 = W * (c + 1) / G;
  const int64_t want = u0 / hr;  // tiles of whole sequences before u0 lie below this
  int64_t before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int L = 0, n = 0, nt = 0;
    if (b0 + lane < p.B) {
      attn_sizes(p, b0 + lane, L, n);
      nt = attn_tiles<TK>(L, n);
    }
    int inc = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, before + inc > want);
    if (past) {
      const int who = __ffs(past) - 1;
      cur.b = b0 + who;
      cur.L = __shfl_sync(0xFFFFFFFFu, L, who);
      cur.n = __shfl_sync(0xFFFFFFFFu, n, who);
      cur.ntiles = __shfl_sync(0xFFFFFFFFu, nt, who);
      before += __shfl_sync(0xFFFFFFFFu, inc - nt, who);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  const int64_t rem = u0 - before * hr;
  const int hrt = (int)(rem / cur.ntiles);
  cur.tile = (int)(rem - (int64_t)hrt * cur.ntiles);
  cur.h = hrt / p.RT;
  cur.rt = hrt - cur.h * p.RT;
  return cur;
}

template <int TK>
__device__ __forceinline__ void attn_next(const AttnParams& p, AttnCursor& c) {
  if (++c.tile < c.ntiles) return;
  c.tile = 0;
  if (++c.rt < p.RT) return;
  c.rt = 0;
  if (++c.h < p.Hkv) return;
  c.h = 0;
  if (++c.b < p.B) {
    attn_sizes(p, c.b, c.L, c.n);
    c.ntiles = attn_tiles<TK>(c.L, c.n);
  }
}

// The CTA that owns unit u.
__device__ __forceinline__ int attn_owner(int64_t u, int64_t W, int G) {
  return (int)(((u + 1) * G - 1) / W);
}

// Whether the item of a worker's last unit goes on in the next worker's range: 0
// no, 1 yes, having begun in this one, 2 yes, having begun before.
__device__ __forceinline__ int attn_cut(bool goes_on, bool began_here) { return goes_on ? (began_here ? 1 : 2) : 0; }

// The weight of a partial sum with maximum m and sum l when it is joined to
// others under the maximum mn: 0 for a part that saw nothing (and not for one
// whose scores were all NaN, which has a NaN sum).
__device__ __forceinline__ float attn_weight(float m, float l, float mn) {
  return m == -INFINITY && l == 0.f ? 0.f : ex2(m - mn);
}

// Which nodes row r of an item sees, as bits; 0 for rows that give zeros.
__device__ __forceinline__ uint64_t attn_bits(const AttnParams& p, int b, int n, int r) {
  const int t = r / p.g;
  if (t >= n) return 0;
  const uint64_t live = n >= 64 ? ~0ull : (1ull << n) - 1;
  const uint64_t m = p.mask ? __ldg(reinterpret_cast<const unsigned long long*>(p.mask) + b * p.ld_mask + t)
                            : (t >= 63 ? ~0ull : (2ull << t) - 1);
  return m & live;
}

// Two packed fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// One thread's four columns of row r (of ROWS) of an item's output.
template <bool BF16>
__device__ __forceinline__ void attn_store4(const AttnParams& p, const AttnCursor& cur, int ro, int c4, float4 a,
                                            float m, float l) {
  const int t = ro / p.g, i = ro - t * p.g;
  const bool live = t < cur.n;
  uint2 v = make_uint2(0u, 0u);
  if (live && l != 0.f) {
    const float iv = 1.f / l;
    v = make_uint2(pack16<BF16>(a.x * iv, a.y * iv), pack16<BF16>(a.z * iv, a.w * iv));
  }
  *reinterpret_cast<uint2*>(p.out + cur.b * p.o_sb + t * p.o_st + (int64_t)(cur.h * p.g + i) * p.o_sh + c4) = v;
  if (p.lse && c4 == 0)
    p.lse[((int64_t)cur.b * p.T + t) * p.Hq + cur.h * p.g + i] =
        live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Which of the 32 cache rows from node t on (cached rows where t < 0) a row with
// node bits `bits` sees.
__device__ __forceinline__ uint32_t attn_seen32(uint64_t bits, int t) {
  if (t >= 64) return 0u;
  if (t >= 0) return (uint32_t)(bits >> t);
  if (t <= -32) return ~0u;
  return (uint32_t)(bits << -t) | ((1u << -t) - 1);
}

}  // namespace qmm
