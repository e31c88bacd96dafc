// qmm_attn_mma.cu -- tree attention for up to 16 rows per key/value head (32 in
// many short sequences), on mma.sync: one pass over the cached rows with a running softmax.
//
// Per row r and cache row j: s = q_r . K_j (m16n8k16, rows as M), then with the
// running maximum m, p = 2^(c s - m), l += p, O += p V_j, all fp32.  m may lag
// behind the true maximum by up to 8 (p <= 2^8; in f16 2^15, ATTN_BASE_BELOW), so
// that O is rescaled only when a row's maximum grows by more than that.
//
// With at most 16 rows there are at most 32 flops for each byte of the cache, so
// the kernel is bound by the cache's stream.  Every warp of the CTA keeps a
// private ring of 16-row blocks of K and V in shared memory (cp.async,
// XOR-swizzled for ldmatrix) and walks its own blocks, every fourth one of the
// CTA's range, without any barrier between warps; the ring runs across the ends
// of segments, so a batch of short sequences streams like one long one.  Barriers
// and shared-memory sums are paid once a segment.
// Where the segments are many and short, every warp takes units and segments of
// its own instead (SOLO; the rule and both sides' times stand at attn_solo).
// Measured: one sequence of 131,071 rows, 20 heads of 128, 16 rows a head, 1.34
// GB: 203 us without the joining kernel (6.6 TB/s, 97 % of a copy), 210 with it;
// 32 sequences of 2,048 to 8,192 rows, 8 rows a head: 115 us (6.1 TB/s).  Two row
// tiles a warp (32 rows) took 103 us where the tcgen05 kernel takes 81 (16 x
// 4096, 20 heads), so 17 rows and more go there.  P is rounded to 16 bits, as the
// product needs it; l sums what was not rounded.  216 registers leave room on the
// SM for the joining kernel beside two CTAs.
#include <cuda.h>
#include <cuda_runtime.h>

#include "qmm_attn.cuh"
#include "qmm_attn.h"

namespace qmm {

namespace {

constexpr int WARPS = 4;
constexpr int BLK = 16;            // cache rows of a warp's block
constexpr int STAGES = 3;
constexpr int ROWS = 16;           // rows of an item's tile

template <int D>
struct Smem {
  static constexpr int BLK_BYTES = BLK * D * 2;             // one of K, V
  static constexpr int STAGE_BYTES = 2 * BLK_BYTES;
  static constexpr int MC = 32;                             // columns summed at a time
  static constexpr int PITCH = MC + 4;
  static constexpr int RING = 0;
  static constexpr int SUM = RING + WARPS * STAGES * STAGE_BYTES;
  static constexpr int ML = SUM + WARPS * ROWS * PITCH * 4;  // m, then l: [warp][row]
  static constexpr int BYTES = ML + 2 * WARPS * ROWS * 4;
};

// SOLO: every warp takes units of its own, of one block each, and ends its
// segments alone; else the CTA's warps share units of four blocks.
template <bool SOLO>
constexpr int UNIT = SOLO ? BLK : WARPS * BLK;

template <bool BF16, int D, bool SOLO>
__global__ void __maxnreg__(216) attn_mma_kernel(const __grid_constant__ AttnParams p) {
  using Op = typename std::conditional<BF16, Bf16Op, F16Op>::type;
  using S = Smem<D>;
  constexpr int TK = UNIT<SOLO>;
  constexpr int CH = D / 8;   // 16-byte chunks of a row
  constexpr int KS = D / 16;  // k steps of q . K
  constexpr int NT = D / 8;   // column tiles of O
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, gt = lane & 3;

  // What the call reads is there, and the last call's partials were read; only
  // then may the joining kernel, which reads the lengths, take its place.
  pdl_wait();
  pdl_trigger();
  int64_t u0, u1;
  const int worker = SOLO ? (int)blockIdx.x * WARPS + warp : (int)blockIdx.x;  // of the p.grid that share the units
  AttnCursor cur = attn_begin<TK>(p, lane, worker, u0, u1);
  if (u0 >= u1) {
    if (lane == 0 && (SOLO || warp == 0)) p.cuts[worker] = make_int4(0, 0, 0, 0);
    return;
  }
  AttnCursor ld = cur;

  const uint32_t ring = smem_u32(smem) + S::RING + warp * STAGES * S::STAGE_BYTES;
  const int64_t head = (int64_t)D << p.page_shift;

  // Request the warp's block of the unit at `c` into ring slot `slot`.
  auto request = [&](const AttnCursor& c, int slot) {
    const int j0 = c.tile * TK + (SOLO ? 0 : warp * BLK);
    const uint32_t dst = ring + slot * S::STAGE_BYTES;
    const uint16_t *kb = p.k_pool, *vb = p.v_pool;
    bool have = false;
    if (j0 < c.L) {
      const int pid = __ldg(p.table + c.b * p.ld_table + (j0 >> p.page_shift));
      have = pid >= 0 && pid < p.n_pages;
      if (have) {
        const int64_t off = pid * p.page_stride + c.h * head + (int64_t)(j0 & ((1 << p.page_shift) - 1)) * D;
        kb += off;
        vb += off;
      } else {
        atomicOr(p.status, DEV_ERR_INDEX);
      }
    }
    if (j0 + BLK <= c.L) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const int id = i * 32 + lane, row = id / CH, ch = id % CH;
        const uint32_t o = row * (D * 2) + ((ch ^ (row & 7)) << 4);
        cp_async16(dst + o, kb + id * 8, have ? 16 : 0);
        cp_async16(dst + S::BLK_BYTES + o, vb + id * 8, have ? 16 : 0);
      }
    } else {
      const uint16_t* kn = p.kn + c.b * p.k_sb + c.h * p.k_sh;
      const uint16_t* vn = p.vn + c.b * p.v_sb + c.h * p.v_sh;
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const int id = i * 32 + lane, row = id / CH, ch = id % CH;
        const int j = j0 + row, t = j - c.L;
        const uint32_t o = row * (D * 2) + ((ch ^ (row & 7)) << 4);
        const bool old = t < 0, fresh = t >= 0 && t < c.n;
        const uint32_t bytes = (old && have) || fresh ? 16 : 0;
        cp_async16(dst + o, fresh ? kn + t * p.k_st + ch * 8 : (bytes ? kb + id * 8 : p.k_pool), bytes);
        cp_async16(dst + S::BLK_BYTES + o, fresh ? vn + t * p.v_st + ch * 8 : (bytes ? vb + id * 8 : p.v_pool),
                   bytes);
      }
    }
  };

  uint32_t qf[KS][4];
  float o[NT][4];
  float m[2], l[2];
  uint64_t bits[2];
  bool fresh_item = true;
  int64_t seg_u = u0;  // first unit of the segment

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (u0 + s < u1) {
      request(ld, s);
      attn_next<TK>(p, ld);
    }
    cp_async_commit();
  }

  int slot = 0, fill = STAGES - 1;
  for (int64_t u = u0; u < u1; ++u) {
    if (u + STAGES - 1 < u1) {
      request(ld, fill);
      attn_next<TK>(p, ld);
    }
    cp_async_commit();
    fill = fill + 1 == STAGES ? 0 : fill + 1;

    if (fresh_item) {
      fresh_item = false;
      seg_u = u;
      const uint16_t* qb = p.q + cur.b * p.q_sb;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = cur.rt * ROWS + half * 8 + gr;
        const bool in = r < p.R;
        const int t = r / p.g, i = r - t * p.g;
        const uint16_t* qr = qb + t * p.q_st + (int64_t)(cur.h * p.g + i) * p.q_sh + gt * 2;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][half] = in ? *reinterpret_cast<const uint32_t*>(qr + ks * 16) : 0u;
          qf[ks][2 + half] = in ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8) : 0u;
        }
        bits[half] = in ? attn_bits(p, cur.b, cur.n, r) : 0;
        m[half] = -INFINITY;
        l[half] = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    }

    cp_async_wait<STAGES - 1>();
    __syncwarp();

    const uint32_t kt = ring + slot * S::STAGE_BYTES, vt = kt + S::BLK_BYTES;
    const int j0 = cur.tile * TK + (SOLO ? 0 : warp * BLK);
    const bool edge = j0 + BLK > cur.L;  // some rows are nodes, or past the end
    unsigned bad = 0;                    // nodes of the block whose V is not finite

    if (edge && j0 < cur.L + cur.n) {
      // Nodes: write their rows to the cache, and take non-finite V out of
      // the product (0 * NaN would reach rows that may not see them).
      const int pid = __ldg(p.table + cur.b * p.ld_table + (j0 >> p.page_shift));
      const bool have = pid >= 0 && pid < p.n_pages;
      if (!have) atomicOr(p.status, DEV_ERR_INDEX);
      const int64_t off = pid * p.page_stride + cur.h * head + (int64_t)(j0 & ((1 << p.page_shift) - 1)) * D;
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        const int id = i * 32 + lane, row = id / CH, ch = id % CH;
        const int t = j0 + row - cur.L;
        const uint32_t so = row * (D * 2) + ((ch ^ (row & 7)) << 4);
        const bool node = t >= 0 && t < cur.n;
        bool nf = false;
        if (node) {
          uint4 kv = lds128(kt + so), vv = lds128(vt + so);
          if (have && cur.rt == 0) {
            *reinterpret_cast<uint4*>(p.k_pool + off + id * 8) = kv;
            *reinterpret_cast<uint4*>(p.v_pool + off + id * 8) = vv;
          }
          nf = any_nonfinite<BF16>(vv);
          if (nf) {
            vv.x = zero_nonfinite<BF16>(vv.x);
            vv.y = zero_nonfinite<BF16>(vv.y);
            vv.z = zero_nonfinite<BF16>(vv.z);
            vv.w = zero_nonfinite<BF16>(vv.w);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(vt + so), "r"(vv.x), "r"(vv.y), "r"(vv.z),
                         "r"(vv.w)
                         : "memory");
          }
        }
        bad |= __reduce_or_sync(0xFFFFFFFFu, nf ? 1u << row : 0u);
      }
      __syncwarp();
    }

    // scores
    float s[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int row = (lane & 7) + ((lane >> 4) << 3);
      const int ch = ks * 2 + ((lane >> 3) & 1);
      uint32_t b0, b1, b2, b3;
      ldmatrix_x4(kt + row * (D * 2) + ((ch ^ (row & 7)) << 4), b0, b1, b2, b3);
      Op::mma(s[0], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1, s[0]);
      Op::mma(s[1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2, b3, s[1]);
    }
    if (edge) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t see = attn_seen32(bits[half], j0 + gt * 2 - cur.L);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!(see >> (nt * 8 + e) & 1)) s[nt][2 * half + e] = -INFINITY;
      }
    }

    // running softmax
    uint32_t pf[4];
    float mx[2];
    bool grow = false;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x = fmaxf(fmaxf(s[0][2 * half], s[0][2 * half + 1]),
                      fmaxf(s[1][2 * half], s[1][2 * half + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
      mx[half] = x * p.scale_log2 - ATTN_BASE_BELOW<BF16>;
      grow |= mx[half] > m[half] + 8.f;
    }
    if (__any_sync(0xFFFFFFFFu, grow)) {
      float a[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float mn = fmaxf(m[half], mx[half]);
        a[half] = m[half] == -INFINITY ? 0.f : ex2(m[half] - mn);
        m[half] = mn;
        l[half] *= a[half];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] *= a[e >> 1];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float base = m[half] == -INFINITY ? 0.f : m[half];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[nt][2 * half + e];
          x = ex2(fmaf(x, p.scale_log2, -base));
          l[half] += x;
        }
    }
    pf[0] = pack16<BF16>(s[0][0], s[0][1]);
    pf[1] = pack16<BF16>(s[0][2], s[0][3]);
    pf[2] = pack16<BF16>(s[1][0], s[1][1]);
    pf[3] = pack16<BF16>(s[1][2], s[1][3]);

    // O += P V
#pragma unroll
    for (int nn = 0; nn < NT / 2; ++nn) {
      const int row = lane & 15, ch = nn * 2 + (lane >> 4);
      uint32_t b0, b1, b2, b3;
      ldmatrix_x4_trans(vt + row * (D * 2) + ((ch ^ (row & 7)) << 4), b0, b1, b2, b3);
      Op::mma(o[2 * nn], pf[0], pf[1], pf[2], pf[3], b0, b1, o[2 * nn]);
      Op::mma(o[2 * nn + 1], pf[0], pf[1], pf[2], pf[3], b2, b3, o[2 * nn + 1]);
    }
    if (bad) {
      // the non-finite values of V, for the rows that see their nodes
      const uint16_t* vn = p.vn + cur.b * p.v_sb + cur.h * p.v_sh;
      for (int jj = 0; jj < BLK; ++jj) {
        if (!(bad >> jj & 1)) continue;
        const int t = j0 + jj - cur.L;
        const int from = (lane & ~3) | ((jj & 7) >> 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float e0 = jj < 8 ? s[0][2 * half] : s[1][2 * half];
          const float e1 = jj < 8 ? s[0][2 * half + 1] : s[1][2 * half + 1];
          const float w = __shfl_sync(0xFFFFFFFFu, jj & 1 ? e1 : e0, from);
          if (bits[half] >> t & 1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v = unpack16<BF16>(__ldg(vn + t * p.v_st + nt * 8 + gt * 2 + e));
                if (!isfinite(v)) o[nt][2 * half + e] += w * v;
              }
          }
        }
      }
    }
    __syncwarp();
    slot = slot + 1 == STAGES ? 0 : slot + 1;

    const bool last_tile = cur.tile + 1 == cur.ntiles;
    if (last_tile || u + 1 == u1) {
      // ------------------------------------------------ end of the segment
      const int64_t item_u = u - cur.tile;  // the item's first unit
      const bool whole = item_u == seg_u && last_tile;
      if (u + 1 == u1 && lane == 0 && (SOLO || warp == 0))
        p.cuts[worker] = make_int4(cur.b, cur.h, cur.rt, attn_cut(!last_tile, item_u >= u0));
      constexpr int PART = ROWS * (D + 2);
      // slot 1: the item begins in this worker's range
      float* part = p.ws + ((int64_t)worker * 2 + (item_u >= u0 ? 1 : 0)) * PART;
      if constexpr (SOLO) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x = l[half];
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
          const int lr = half * 8 + gr, r = cur.rt * ROWS + lr;
          if (whole) {
            const int t = r / p.g, i = r - t * p.g;
            if (r >= p.R) continue;
            const bool live = t < cur.n;
            const float inv = live && x != 0.f ? 1.f / x : 0.f;
            uint16_t* to = p.out + cur.b * p.o_sb + t * p.o_st + (int64_t)(cur.h * p.g + i) * p.o_sh + gt * 2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              *reinterpret_cast<uint32_t*>(to + nt * 8) =
                  inv != 0.f ? pack16<BF16>(o[nt][2 * half] * inv, o[nt][2 * half + 1] * inv) : 0u;
            if (p.lse && gt == 0)
              p.lse[((int64_t)cur.b * p.T + t) * p.Hq + cur.h * p.g + i] =
                  live ? (m[half] + log2f(x)) * 0.69314718055994531f : -INFINITY;
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              *reinterpret_cast<float2*>(part + lr * D + nt * 8 + gt * 2) =
                  make_float2(o[nt][2 * half], o[nt][2 * half + 1]);
            if (gt == 0) {
              part[ROWS * D + lr] = m[half];
              part[ROWS * D + ROWS + lr] = x;
            }
          }
        }
        fresh_item = true;
      } else {
        float* s_ml = reinterpret_cast<float*>(smem + S::ML);
        float* s_sum = reinterpret_cast<float*>(smem + S::SUM);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x = l[half];
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
          if (gt == 0) {
            const int r = half * 8 + gr;
            s_ml[warp * ROWS + r] = m[half];
            s_ml[(WARPS + warp) * ROWS + r] = x;
          }
        }
        __syncthreads();
        float f[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = half * 8 + gr;
          float mn = -INFINITY;
#pragma unroll
          for (int w = 0; w < WARPS; ++w) mn = fmaxf(mn, s_ml[w * ROWS + r]);
          f[half] = attn_weight(m[half], s_ml[(WARPS + warp) * ROWS + r], mn);
        }
        // each thread sums one float4 of a column block over the warps
        const int cr = tid / (S::MC / 4), cc = (tid % (S::MC / 4)) * 4;
        float cm = -INFINITY, cl = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) cm = fmaxf(cm, s_ml[w * ROWS + cr]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float lw = s_ml[(WARPS + w) * ROWS + cr];
          cl += lw * attn_weight(s_ml[w * ROWS + cr], lw, cm);
        }
        const int r_out = cur.rt * ROWS + cr;
        const int t_out = r_out / p.g, i_out = r_out - t_out * p.g;
        const bool in_out = r_out < p.R, live_out = in_out && t_out < cur.n;
        uint16_t* orow = p.out + cur.b * p.o_sb + t_out * p.o_st + (int64_t)(cur.h * p.g + i_out) * p.o_sh;
        const float inv = live_out && cl != 0.f ? 1.f / cl : 0.f;
#pragma unroll
        for (int blk = 0; blk < D / S::MC; ++blk) {
#pragma unroll
          for (int k = 0; k < S::MC / 8; ++k) {
            const int nt = blk * (S::MC / 8) + k;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int r = half * 8 + gr;
              float2 v = make_float2(o[nt][2 * half] * f[half], o[nt][2 * half + 1] * f[half]);
              *reinterpret_cast<float2*>(s_sum + (warp * ROWS + r) * S::PITCH + k * 8 + gt * 2) = v;
            }
          }
          __syncthreads();
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(s_sum + (w * ROWS + cr) * S::PITCH + cc);
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
          }
          if (!whole) {
            *reinterpret_cast<float4*>(part + cr * D + blk * S::MC + cc) = a;
          } else if (in_out) {
            uint2 v = make_uint2(0u, 0u);
            if (inv != 0.f) v = make_uint2(pack16<BF16>(a.x * inv, a.y * inv), pack16<BF16>(a.z * inv, a.w * inv));
            *reinterpret_cast<uint2*>(orow + blk * S::MC + cc) = v;
          }
          __syncthreads();
        }
        if (whole) {
          if (p.lse && in_out && cc == 0)
            p.lse[((int64_t)cur.b * p.T + t_out) * p.Hq + cur.h * p.g + i_out] =
                live_out ? (cm + log2f(cl)) * 0.69314718055994531f : -INFINITY;
        } else {
          if (cc == 0) {
            part[ROWS * D + cr] = cm;
            part[ROWS * D + ROWS + cr] = cl;
          }
        }
        __syncthreads();
        fresh_item = true;
      }
    }
    attn_next<TK>(p, cur);
  }
  cp_async_wait<0>();
}

template <bool BF16, int D, bool SOLO>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_mma_kernel<BF16, D, SOLO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem<D>::BYTES);
}

template <bool BF16, int D, bool SOLO>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SOLO ? p.grid / WARPS : p.grid));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = Smem<D>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_mma_kernel<BF16, D, SOLO>, p);
}

template <bool BF16, int D>
cudaError_t prepare_both() {
  const cudaError_t e = prepare<BF16, D, true>();
  return e == cudaSuccess ? prepare<BF16, D, false>() : e;
}

template <bool BF16, int D>
cudaError_t launch_one(const AttnParams& p, bool solo, cudaStream_t st) {
  return solo ? launch<BF16, D, true>(p, st) : launch<BF16, D, false>(p, st);
}

}  // namespace

int attn_mma_tile_cache_rows(bool solo) { return solo ? UNIT<true> : UNIT<false>; }
int attn_mma_tile_rows() { return ROWS; }
int attn_mma_workers(int sms, bool solo) { return sms * ATTN_MMA_CTAS_PER_SM * (solo ? WARPS : 1); }

cudaError_t prepare_attn_mma(bool bf16, int D) {
  if (D == 128) return bf16 ? prepare_both<true, 128>() : prepare_both<false, 128>();
  return bf16 ? prepare_both<true, 64>() : prepare_both<false, 64>();
}

cudaError_t launch_attn_mma(const AttnParams& p, bool bf16, int D, bool solo, cudaStream_t st) {
  if (D == 128) return bf16 ? launch_one<true, 128>(p, solo, st) : launch_one<false, 128>(p, solo, st);
  return bf16 ? launch_one<true, 64>(p, solo, st) : launch_one<false, 64>(p, solo, st);
}

}  // namespace qmm
