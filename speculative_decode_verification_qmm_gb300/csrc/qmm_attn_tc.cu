// qmm_attn_tc.cu -- tree attention for more than 16 rows per key/value head (but
// for 17 to 32 in many short sequences, see attn_solo), on
// the tcgen05 tensor cores: one pass over the cached rows with a running
// softmax.
//
// A CTA takes NQ = 1 or 2 row tiles of 128 rows and walks its range of cache
// tiles of 128 rows.  Per row tile and cache tile:
//   S = Q K^T     M = 128 rows, N = 128 cache rows; Q and K in shared memory
//   P = 2^(c S - m)  with the row's running maximum m, l += P
//   O += P V      A = P in tensor memory (16 bits), B = V in shared memory
// with S, O and the statistics in fp32.  One thread owns one row (a lane of
// tensor memory), so the softmax needs no exchange between threads.  m may lag
// behind the true maximum by up to 8 (P <= 2^8; in f16 2^15, ATTN_BASE_BELOW): O is
// rescaled, by the softmax warps and through their registers, only when a row of
// the warp grows more.
//   warps 0 .. 4 NQ - 1   softmax, rescaling, output (four warps a row tile)
//   two warps (NQ = 2: one) issue the MMAs
//   two warps             load K and V tiles, one ring each: tensor copies of 16
//                         rows, which lie in one page; cp.async for the tree's
//                         nodes, from the caller's rows (and on to the cache), and
//                         the rows around them; Q, once a segment, by both
// Why this split.  At 128 rows a tile of K and V (64 KB) takes 1.5 us of an
// SM's share of the HBM stream, and its two products 0.55 us of the tensor cores
// and its softmax of 16,384 scores 0.8: with one row tile the stream is the
// bound, and S is double-buffered so that Q K^T of the next tile runs under the
// softmax.  One warp then issues all Q K^T, another all P V: the issue of an MMA
// blocks until the one before it is nearly done, and a product whose operands are
// ready would wait behind one whose are not.
// With two row tiles each tile of K and V serves 256 rows, and tensor memory (512
// columns) holds one S and O of each.  One warp issues everything: P V of a row
// tile and, when that has ended, Q K^T of its next cache tile, whose S lies where P
// did, then the same for the other row tile, whose softmax ran meanwhile.  (MMAs with
// different accumulators have no promised order, so the wait is needed; without it
// the case below took 120 us.)  The softmax hands P over in two steps of SW columns, so
// that P V of the first runs under the softmax of the second; a step's P
// overwrites the first half of its S.  Q K^T over all 128 columns at once: over
// 64 it takes as long.  Before, two issuers and S in two buffers of 64 columns
// took 130 us for 4 sequences x 16,384 rows, 64 nodes, 64 heads on 8; this takes
// 126 us (1,097 TFLOP/s; 1,700 cycles a row tile and cache tile, of which the tensor
// cores work 1,024: a softmax of 1,500 cycles and its hand-overs do not fit under
// the other row tile's products.  Two softmax warps a row, half of the columns
// each, need 96 registers a thread, spilled, and took 231 us).
// With one row tile, 64/8 heads: 16 x 8,192 rows, 128 rows a head: 107 us (645
// TFLOP/s, 5.1 TB/s); one sequence of 131,072, 64 rows a head: 91 us (5.9 TB/s).
// P is rounded to 16 bits, as the product needs it; l sums what was not rounded.
// Every wait is bounded; on a timeout the CTA records it, its roles run out of
// their loops without waiting, its copies and MMAs in flight are drained and
// tensor memory is freed.
#include <cuda.h>
#include <cuda_runtime.h>

#include "qmm_attn.cuh"
#include "qmm_attn.h"
#include "qmm_tc.cuh"

namespace qmm {

namespace {

constexpr int TK = 128;   // cache rows of a tile
constexpr int BAD_BUFS = 16;  // more than twice the segments that the rings hold

template <int D, int NQ>
struct Smem {
  static constexpr int TILE = TK * D * 2;           // one of K, V; also 128 rows of Q
  static constexpr int HALF = TK * 128;             // 64 columns of a tile
  static constexpr int KS = D == 128 ? 3 : 4;       // ring of K tiles
  static constexpr int VS = D == 128 ? 4 - NQ : 4;  // ring of V tiles
  static constexpr int Q = 0;
  static constexpr int K = Q + NQ * TILE;
  static constexpr int V = K + KS * TILE;
  static constexpr int BAR = V + VS * TILE;
  // kfull[KS], kempty[KS], vfull[VS], vempty[VS], qfull, qempty, sfull[4],
  // sfree[4], pfull[4], odone[2], olast[2], oempty[2], drain
  static constexpr int NBAR = 2 * (KS + VS) + 21;
  static constexpr int BAD = BAR + NBAR * 8;        // nodes with non-finite V, by segment
  static constexpr int FLAG = BAD + BAD_BUFS * 8;   // [0] abort, [1] tensor memory
  static constexpr int BYTES = FLAG + 16;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// Shared-memory operands, 128-byte swizzle, as the two words of a matrix
// descriptor: the upper word is the same for all (8-row groups 1024 bytes apart,
// version 1, layout type 2), the lower one holds the start address / 16 and, for
// an operand whose rows along K are 128 bytes of 64 consecutive M or N values,
// the distance of the next 64 values / 16.  A step along K adds a constant to
// it, which keeps the issuing thread short: with descriptors built anew for each
// MMA it took 180 cycles to issue one that the tensor cores run in 64.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

// D[tmem] (+)= A * B, kind::f16, fp32 accumulate; A in shared or tensor memory, B in shared.
__device__ __forceinline__ void mma_ss(uint32_t d_t, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_t),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_t, uint32_t a_t, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_t),
      "r"(a_t), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
      : "memory");
}

// Bounded wait that also gives up when another role did.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t lim, volatile int* abort) {
  if (lim == 0) return false;
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  const long long limit = (long long)(lim < (1ull << 40) ? lim : (1ull << 40)) * 2;
  while (!mbar_try_wait(bar, parity)) {
    if (*abort || clock64() - t0 > limit) return false;
  }
  return true;
}

template <bool BF16, int D, int NQ>
__global__ void __launch_bounds__(NQ * 128 + 64 / NQ + 64, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D, NQ>;
  constexpr int ROWS = NQ * 128;
  constexpr int SW = TK / NQ, SUB = TK / SW;  // columns of a step's P, steps of a tile
  constexpr int NB = 2 / NQ;                  // buffers of S of a row tile
  constexpr uint32_t IDESC_S = tc_idesc_n(BF16 ? 1u : 0u, TK);
  constexpr uint32_t IDESC_O = tc_idesc_n(BF16 ? 1u : 0u, D) | (1u << 16);  // B along N
  // tensor memory columns: NB times S, then O, of each row tile
  constexpr uint32_t COL_O = NB * TK;
  constexpr uint32_t COL_Q = 256;  // of the second row tile
  constexpr int MMA_WARP = NQ * 4, MMA_WARPS = 2 / NQ, LOAD_WARP = MMA_WARP + MMA_WARPS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t b_kfull = base + S::BAR, b_kempty = b_kfull + S::KS * 8, b_vfull = b_kempty + S::KS * 8,
                 b_vempty = b_vfull + S::VS * 8, b_qfull = b_vempty + S::VS * 8, b_qempty = b_qfull + 8,
                 b_sfull = b_qempty + 8, b_sfree = b_sfull + 32, b_pfull = b_sfree + 32, b_odone = b_pfull + 32,
                 b_olast = b_odone + 16, b_oempty = b_olast + 16, b_drain = b_oempty + 16;  // sfull, sfree, pfull: [row tile][buffer]
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + S::FLAG);
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(smem + S::BAD);

  if (tid == 0) {
    for (int i = 0; i < S::KS; ++i) {
      mbar_init(b_kfull + 8 * i, 1);
      mbar_init(b_kempty + 8 * i, 1);
    }
    for (int i = 0; i < S::VS; ++i) {
      mbar_init(b_vfull + 8 * i, 1);
      mbar_init(b_vempty + 8 * i, 1);
    }
    mbar_init(b_qfull, 2);
    mbar_init(b_qempty, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_sfree + 8 * i, 1);
      mbar_init(b_pfull + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_odone + 8 * i, 1);
      mbar_init(b_olast + 8 * i, 1);
      mbar_init(b_oempty + 8 * i, 4);
    }
    mbar_init(b_drain, MMA_WARPS);
    for (int i = 0; i < BAD_BUFS; ++i) s_bad[i] = 0;
    s_flag[0] = 0;
    if (base & 1023u) {
      atomicOr(p.status, DEV_ERR_SMEM_ALIGN);
      s_flag[0] = 1;
    }
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(base + S::FLAG + 4, 512);
  // What the call reads is there, and the last call's partials were read; only
  // then may the joining kernel, which reads the lengths, take its place.
  pdl_wait();
  pdl_trigger();
  int64_t u0, u1;
  AttnCursor cur = attn_begin<TK>(p, lane, blockIdx.x, u0, u1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, (uint32_t)s_flag[1], 0);

  if (tid == 0 && u0 >= u1) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  const uint64_t lim = p.wait_limit_ns;
  auto fail = [&](int code) {
    if (!s_flag[0]) atomicOr(p.status, code);
    s_flag[0] = 1;
  };
  // The cache tiles of the segment that starts at unit u.
  auto segment = [&](int64_t u) {
    const int64_t left = cur.ntiles - cur.tile;
    return (int)(left < u1 - u ? left : u1 - u);
  };

  if (warp >= LOAD_WARP) {
    // ------------------------------------------------------------ load
    const bool is_v = warp > LOAD_WARP;
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    const uint32_t full = is_v ? b_vfull : b_kfull, empty = is_v ? b_vempty : b_kempty;
    const uint32_t ring = base + (is_v ? S::V : S::K);
    const int slots = is_v ? S::VS : S::KS;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    uint16_t* pool = is_v ? p.v_pool : p.k_pool;
    const int64_t head = (int64_t)D << p.page_shift;
    constexpr int BLOCKS = TK / 16;  // 16 rows, one tensor copy a half
    bool ok = s_flag[0] == 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xFFFFFFFFu, ok && wait_or_abort(bar, parity, lim, s_flag));
      if (!ok && lane == 0) fail(DEV_ERR_TIMEOUT_EMPTY);
    };
    auto hand_on = [&](uint32_t bar) {
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int slot = 0, round = 0, seg = 0;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      const int count = segment(u);
      // Q, by both warps; rows past the item's stay as they are, and so do their results
      if (seg > 0) wait(b_qempty, (uint32_t)((seg - 1) & 1));
      if (!ok) break;
      const int rows = p.R - cur.rt * ROWS < ROWS ? p.R - cur.rt * ROWS : ROWS;
      {
        constexpr int STEP = 64 / CH;  // rows of both warps at a time
        const int id = (warp - LOAD_WARP) * 32 + lane, ch = id % CH;
        const int dt = STEP / p.g, dh = STEP % p.g;
        int row = id / CH, t = (cur.rt * ROWS + row) / p.g, h = (cur.rt * ROWS + row) % p.g;
        const uint16_t* src = p.q + cur.b * p.q_sb + (int64_t)cur.h * p.g * p.q_sh + ch * 8;
#pragma unroll 4
        for (; row < rows; row += STEP) {
          cp_async16(base + S::Q + (row >> 7) * S::TILE + (ch >> 3) * S::HALF + (row & 127) * 128 +
                         (((ch & 7) ^ (row & 7)) << 4),
                     src + t * p.q_st + h * p.q_sh, 16);
          t += dt, h += dh;
          if (h >= p.g) h -= p.g, ++t;
        }
      }
      // Lane i < BLOCKS looks up the page of the tile's block i, a tile ahead.  An
      // id out of range is reported; rows of page 0 take its place, unwritten.
      int ahead = 0;
      auto lookup = [&](int j) {
        const int jb = j * TK + lane * 16;
        ahead = 0;
        if (lane < BLOCKS && jb < cur.L + cur.n) {
          ahead = __ldg(p.table + cur.b * p.ld_table + (jb >> p.page_shift));
          if (ahead < 0 || ahead >= p.n_pages) {
            atomicOr(p.status, DEV_ERR_INDEX);
            ahead = -1;
          }
        }
      };
      lookup(cur.tile);
      hand_on(b_qfull);
      for (int j = 0; j < count; ++j) {
        const int j0 = (cur.tile + j) * TK;
        const int pid = ahead;
        if (j + 1 < count) lookup(cur.tile + j + 1);
        if (round > 0) wait(empty + 8 * slot, (uint32_t)((round - 1) & 1));
        if (!ok) break;
        const uint32_t bar = full + 8 * slot, dst = ring + slot * S::TILE;
        // blocks that hold cached rows only
        int whole = cur.L > j0 ? (cur.L - j0) / 16 : 0;
        whole = whole < BLOCKS ? whole : BLOCKS;
        if (lane == 0) {
          if (whole == BLOCKS)
            mbar_arrive_expect_tx(bar, S::TILE);
          else if (whole > 0)
            mbar_expect_tx(bar, whole * 16 * D * 2);
        }
        __syncwarp();
        if (lane < whole) {
          const int64_t row = p.row0 + (((int64_t)(pid < 0 ? 0 : pid) * p.Hkv + cur.h) << p.page_shift) +
                              ((j0 + lane * 16) & ((1 << p.page_shift) - 1));
#pragma unroll
          for (int half = 0; half < D / 64; ++half)
            tma_load_2d(dst + half * S::HALF + lane * 2048, map, half * 64, (int)row, bar);
        }
        if (whole < BLOCKS) {
          const uint16_t* fresh = is_v ? p.vn + cur.b * p.v_sb + cur.h * p.v_sh : p.kn + cur.b * p.k_sb + cur.h * p.k_sh;
          const int64_t fresh_st = is_v ? p.v_st : p.k_st;
          const int end = cur.L + cur.n - j0;  // rows of the tile that exist
#pragma unroll 1
          for (int blk = whole; blk < BLOCKS; ++blk) {
            const int id0 = __shfl_sync(0xFFFFFFFFu, pid, blk);
            const uint16_t* from = pool + (id0 < 0 ? 0 : id0) * p.page_stride + cur.h * head +
                                   (int64_t)((j0 + blk * 16) & ((1 << p.page_shift) - 1)) * D;
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              const int id = i * 32 + lane, row = blk * 16 + id / CH, ch = id % CH;
              const int t = j0 + row - cur.L;
              const bool node = t >= 0 && t < cur.n;
              const uint32_t bytes = node || (t < 0 && id0 >= 0) ? 16 : 0;
              const uint16_t* src = node ? fresh + t * fresh_st + ch * 8 : (bytes ? from + id * 8 : pool);
              cp_async16(dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4), src, bytes);
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          // Nodes: on to the cache, and non-finite V out of the product.  A
          // lane reads back the chunks that it requested.
          for (int blk = whole; blk < BLOCKS && blk * 16 < end; ++blk) {
            const int id0 = __shfl_sync(0xFFFFFFFFu, pid, blk);
            uint16_t* to = pool + (id0 < 0 ? 0 : id0) * p.page_stride + cur.h * head +
                           (int64_t)((j0 + blk * 16) & ((1 << p.page_shift) - 1)) * D;
            uint4 v[CH / 2];
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              const int id = i * 32 + lane, row = blk * 16 + id / CH, ch = id % CH;
              v[i] = lds128(dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            }
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              const int id = i * 32 + lane, row = blk * 16 + id / CH, ch = id % CH;
              const int t = j0 + row - cur.L;
              if (t < 0 || t >= cur.n) continue;
              if (id0 >= 0 && cur.rt == 0) *reinterpret_cast<uint4*>(to + id * 8) = v[i];
              if (is_v && any_nonfinite<BF16>(v[i])) {
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                 dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4)),
                             "r"(zero_nonfinite<BF16>(v[i].x)), "r"(zero_nonfinite<BF16>(v[i].y)),
                             "r"(zero_nonfinite<BF16>(v[i].z)), "r"(zero_nonfinite<BF16>(v[i].w))
                             : "memory");
                atomicOr(s_bad + (seg & (BAD_BUFS - 1)), 1ull << t);
              }
            }
          }
          hand_on(bar);
        }
        if (++slot == slots) slot = 0, ++round;
      }
      cur.tile += count - 1;
      attn_next<TK>(p, cur);
      u += count;
    }
    cp_async_wait<0>();
    // Tensor copies in flight land before the CTA leaves: the last tile of every
    // slot.  Always: another role can give up after this one's last look at the flag.
    for (int i = 0; i < slots; ++i) {
      const int rounds = i < slot ? round + 1 : round;
      if (rounds > 0 && lane == 0 && !mbar_wait_bounded(full + 8 * i, (rounds - 1) & 1, 1000000000ull))
        atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
    }
  } else if (warp >= MMA_WARP) {
    // ------------------------------------------------------------ MMA issue
    // The warp stays together and one elected lane issues: operands then live in
    // uniform registers, and an MMA costs 48 to 64 cycles to issue, what it
    // takes to run; from a branch on the lane it was 63 alone and above 130
    // beside two softmax warps.
    {
      uint32_t leader;
      asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
      const int who = warp - MMA_WARP;  // 0: Q K^T, 1: P V
      bool ok = s_flag[0] == 0;
      auto need = [&](uint32_t bar, int phase) {
        if (ok && !__all_sync(0xFFFFFFFFu, wait_or_abort(bar, (uint32_t)(phase & 1), lim, s_flag))) {
          if (leader) fail(DEV_ERR_TIMEOUT_FULL);
          ok = false;
        }
        return ok;
      };
      // S of row tile q and the K tile in `slot`, into column d
      auto product_s = [&](int q, int slot, uint32_t d) {
        const uint32_t a = desc_lo(base + S::Q + q * S::TILE), b = desc_lo(base + S::K + slot * S::TILE);
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (uint32_t)(kk >> 2) * (S::HALF >> 4) + (uint32_t)(kk & 3) * (32 >> 4);
            mma_ss(d, a + o, b + o, IDESC_S, kk > 0);
          }
        }
      };
      // O of row tile q += P of a step (its part of the V tile in `slot`)
      auto product_o = [&](int q, int slot, int step, bool first) {
        const uint32_t a = tmem + q * COL_Q + (step & 1) * SW, d = tmem + q * COL_Q + COL_O;
        const uint32_t b = desc_lo_mn(base + S::V + slot * S::TILE + step % SUB * SW * 128, S::HALF);
        tc_fence_after();
        if (leader) {
          mma_ts(d, a, b, IDESC_O, !first);
#pragma unroll
          for (int kk = 1; kk < SW / 16; ++kk) mma_ts(d, a + kk * 8, b + kk * (2048 >> 4), IDESC_O, 1);
          tc_commit(b_odone + 8 * q);
        }
      };
      int n = 0, seg = 0;          // tiles and segments so far (n: parities, and whether there was one)
      int slot = 0, round = 0;     // of the tile of K or V
      int vslot = 0, vround = 0;   // of the tile of V, where one warp issues both
      for (int64_t u = u0; u < u1 && ok; ++seg) {
        const int count = segment(u);
        if constexpr (NQ == 2) {
          // O += P V of a row tile, then S of its next tile, then the other row tile
          for (int j = -1; j < count && ok; ++j) {
            if (j < 0 && !need(b_qfull, seg)) break;
            for (int q = 0; q < 2 && ok; ++q) {
              if (j >= 0) {
                if (q == 0 && !need(b_vfull + 8 * vslot, vround)) break;
                if (j == 0 && seg > 0 && !need(b_oempty + 8 * q, seg - 1)) break;
#pragma unroll
                for (int sub = 0; sub < SUB; ++sub) {
                  if (!need(b_pfull + 8 * (2 * q + sub), n)) break;
                  product_o(q, vslot, sub, j == 0 && sub == 0);
                }
                if (!ok) break;
                if (leader) tc_commit(b_sfree + 8 * q);
                if (leader && j + 1 == count) tc_commit(b_olast + 8 * q);
              }
              if (j + 1 < count) {
                if (q == 0 && !need(b_kfull + 8 * slot, round)) break;
                // S goes where P of the tile before lies, until its products have ended
                const int before = j >= 0 ? n : n - 1;
                if (before >= 0 && !need(b_sfree + 8 * q, before)) break;
                product_s(q, slot, tmem + q * COL_Q);
                if (leader) tc_commit(b_sfull + 8 * (2 * q));
              }
            }
            if (!ok) break;
            if (j >= 0) {
              if (leader) tc_commit(b_vempty + 8 * vslot);
              if (++vslot == S::VS) vslot = 0, ++vround;
              ++n;
            }
            if (j + 1 < count) {
              if (leader) tc_commit(b_kempty + 8 * slot);
              if (leader && j + 2 == count) tc_commit(b_qempty);
              if (++slot == S::KS) slot = 0, ++round;
            }
          }
        } else if (who == 0) {
          if (!need(b_qfull, seg)) break;
          for (int j = 0; j < count; ++j, ++n) {
            if (!need(b_kfull + 8 * slot, round)) break;
            // its S held P of two tiles ago until the product of that was done
            if (n >= 2 && !need(b_sfree + 8 * (n & 1), (n >> 1) - 1)) break;
            product_s(0, slot, tmem + (n & 1) * TK);
            if (leader) tc_commit(b_sfull + 8 * (n & 1));
            if (leader) tc_commit(b_kempty + 8 * slot);
            if (leader && j + 1 == count) tc_commit(b_qempty);
            if (++slot == S::KS) slot = 0, ++round;
          }
        } else {
          for (int j = 0; j < count; ++j, ++n) {
            if (!need(b_vfull + 8 * slot, round) || !need(b_pfull + 8 * (n & 1), n >> 1)) break;
            if (j == 0 && seg > 0 && !need(b_oempty, seg - 1)) break;
            product_o(0, slot, n, j == 0);
            if (leader) tc_commit(b_sfree + 8 * (n & 1));
            if (leader && j + 1 == count) tc_commit(b_olast);
            if (leader) tc_commit(b_vempty + 8 * slot);
            if (++slot == S::VS) slot = 0, ++round;
          }
        }
        cur.tile += count - 1;
        attn_next<TK>(p, cur);
        u += count;
      }
      // all MMAs of the CTA have ended before tensor memory is given back
      if (leader) {
        tc_commit(b_drain);
        if (!mbar_wait_bounded(b_drain, 0, 1000000000ull)) atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + q * COL_Q;
    const uint32_t t_o = tl + COL_O;
    bool ok = s_flag[0] == 0;
    auto need = [&](uint32_t bar, int phase) {
      if (ok) {
        const bool got = __all_sync(0xFFFFFFFFu, wait_or_abort(bar, (uint32_t)(phase & 1), lim, s_flag));
        if (!got) {
          if (lane == 0) fail(DEV_ERR_TIMEOUT_FULL);
          ok = false;
        }
      }
      return ok;
    };
    int done = 0, seg = 0;  // done: parities only
    for (int64_t u = u0; u < u1; ++seg) {
      const int count = segment(u);
      const int r = cur.rt * ROWS + q * 128 + row;
      const bool in = r < p.R, idle = r - lane >= p.R;
      const uint64_t bits = in ? attn_bits(p, cur.b, cur.n, r) : 0;
      float m = -INFINITY, l = 0.f;
      const int steps = count * SUB;
      for (int j = 0; j < steps; ++j) {
        const int n = done + j;
        const int buf = 2 * q + (n & 1);
        const uint32_t t_s = tl + (n & 1) * SW;
        if (n % SUB == 0) need(b_sfull + 8 * (2 * q + n / SUB % NB), n / SUB / NB);
        if (!ok) continue;
        if (idle) {  // no row of the warp is the item's: whatever P is, nobody looks
          if (lane == 0) mbar_arrive(b_pfull + 8 * buf);
          continue;
        }
        tc_fence_after();
        const int t0 = cur.tile * TK + j * SW - cur.L;  // node of the step's first row, if it is one
        const bool edge = t0 + SW > 0;
        uint32_t v[SW / 32][32];  // the row's scores
#pragma unroll
        for (int c = 0; c < SW / 32; ++c) tmem_ld32(t_s + c * 32, v[c]);
        tmem_wait_ld();
        if (edge) {
#pragma unroll
          for (int c = 0; c < SW / 32; ++c) {
            const uint32_t see = attn_seen32(bits, t0 + c * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1)) v[c][i] = 0xFF800000u;  // -inf
          }
        }
        float mx;
        {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < SW / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              x[(i >> 1) & 3] = fmaxf(x[(i >> 1) & 3], fmaxf(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])));
          mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        }
        mx = mx * p.scale_log2 - ATTN_BASE_BELOW<BF16>;
        // (rows past the item's hold anything and must not decide for the others)
        if (__any_sync(0xFFFFFFFFu, in && mx > m + 8.f)) {
          const float mn = fmaxf(m, mx);
          const float a = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= a;
          if (j > 0) {
            // a parity tells a phase from the next one only: the product before
            // the last was done when this S was computed
            if (!need(b_odone + 8 * q, n - 1)) continue;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t x[16];
              tmem_ld16(t_o + c * 16, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * a);
              tmem_st16(t_o + c * 16, x);
            }
          }
        }
        const float mb = m == -INFINITY ? 0.f : m;
        const float2 c2 = make_float2(p.scale_log2, p.scale_log2), m2 = make_float2(-mb, -mb);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < SW / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 e = fma2(make_float2(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), c2, m2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], e);
            w[i / 2] = pack16<BF16>(e.x, e.y);
          }
          tmem_st16(t_s + c * 16, w);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_pfull + 8 * buf);
      }

      // ------------------------------------------------ end of the segment
      need(b_olast + 8 * q, seg);
      tc_fence_after();
      const int64_t item_u = u - cur.tile;  // the item's first unit
      const bool last_tile = cur.tile + count == cur.ntiles;
      const bool whole = cur.tile == 0 && last_tile;
      if (tid == 0 && u + count == u1)
        p.cuts[blockIdx.x] = make_int4(cur.b, cur.h, cur.rt, attn_cut(!last_tile, item_u >= u0));
      constexpr int PART = ROWS * (D + 2);
      float* part = p.ws + ((int64_t)blockIdx.x * 2 + (item_u >= u0 ? 1 : 0)) * PART;
      const int t_row = r / p.g, i_row = r - t_row * p.g;
      const bool live = in && t_row < cur.n;
      const unsigned long long bad = s_bad[seg & (BAD_BUFS - 1)];
      if (tid == 0) s_bad[(seg + BAD_BUFS / 2) & (BAD_BUFS - 1)] = 0;  // read by all, not yet written again
      auto write16 = [&](int t, int i, int c, const float (&a)[32], float inv) {
        uint16_t* to = p.out + cur.b * p.o_sb + t * p.o_st + (int64_t)(cur.h * p.g + i) * p.o_sh + c;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint4 o = make_uint4(0u, 0u, 0u, 0u);
          if (inv != 0.f)
            o = make_uint4(pack16<BF16>(a[k] * inv, a[k + 1] * inv), pack16<BF16>(a[k + 2] * inv, a[k + 3] * inv),
                           pack16<BF16>(a[k + 4] * inv, a[k + 5] * inv), pack16<BF16>(a[k + 6] * inv, a[k + 7] * inv));
          *reinterpret_cast<uint4*>(to + k) = o;
        }
      };
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(t_o + c, v);
        tmem_wait_ld();
        float a[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(v[i]);
        if (bad) {
          // the non-finite values of V, for the rows that see their nodes
          for (unsigned long long left_bad = bad & bits; left_bad; left_bad &= left_bad - 1) {
            const int t = __ffsll((long long)left_bad) - 1;
            const uint16_t* qr = p.q + cur.b * p.q_sb + t_row * p.q_st + (int64_t)(cur.h * p.g + i_row) * p.q_sh;
            const uint16_t* kr = p.kn + cur.b * p.k_sb + cur.h * p.k_sh + t * p.k_st;
            const uint16_t* vr = p.vn + cur.b * p.v_sb + cur.h * p.v_sh + t * p.v_st + c;
            float s = 0.f;
            for (int d = 0; d < D; ++d) s = fmaf(unpack16<BF16>(qr[d]), unpack16<BF16>(kr[d]), s);
            const float w = ex2(fmaf(s, p.scale_log2, -(m == -INFINITY ? 0.f : m)));
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = unpack16<BF16>(vr[i]);
              if (!isfinite(x)) a[i] += w * x;
            }
          }
        }
        if (!ok || idle) continue;
        if (whole) {
          if (in) write16(t_row, i_row, c, a, inv);
          continue;
        }
        // Eight lanes exchange their rows' 32 columns, so that they store a row at
        // a time, four columns each: a lane's own row, 16 bytes a lane and line,
        // took 8,600 cycles a segment of 256 rows.  (Whole items are 16 bits a
        // value and most often short; there the exchange costs more than it saves:
        // 32 sequences of up to 200 rows, 32 rows a head, 65 us instead of 49.)
#pragma unroll
        for (int h = 4; h > 0; h >>= 1)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!(k & h))
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float &lo = a[k * 4 + e], &hi = a[(k | h) * 4 + e];
                const float x = __shfl_xor_sync(0xFFFFFFFFu, lane & h ? lo : hi, h);
                (lane & h ? lo : hi) = x;
              }
        float* to = part + (q * 128 + (row & ~7)) * D + c + (lane & 7) * 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(to + k * D) = make_float4(a[k * 4], a[k * 4 + 1], a[k * 4 + 2], a[k * 4 + 3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_oempty + 8 * q);
      if (whole) {
        if (ok && in && p.lse)
          p.lse[((int64_t)cur.b * p.T + t_row) * p.Hq + cur.h * p.g + i_row] =
              live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      } else if (ok) {
        part[ROWS * D + q * 128 + row] = m;
        part[ROWS * D + ROWS + q * 128 + row] = l;
      }
      done += steps;
      cur.tile += count - 1;
      attn_next<TK>(p, cur);
      u += count;
    }
  }

  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool BF16, int D, int NQ>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_tc_kernel<BF16, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Smem<D, NQ>::BYTES);
}

template <bool BF16, int D, int NQ>
cudaError_t launch(const AttnParams& p, const void* kmap, const void* vmap, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(NQ * 128 + 64 / NQ + 64);
  cfg.dynamicSmemBytes = Smem<D, NQ>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tc_kernel<BF16, D, NQ>, p, *static_cast<const CUtensorMap*>(kmap),
                            *static_cast<const CUtensorMap*>(vmap));
}

}  // namespace

int attn_tc_tile_cache_rows() { return TK; }
// One row tile of 128 or two.  Two read K and V once for 256 rows, one has S
// double-buffered and its idle warps cost less.  Measured, one against two, in us:
// 128 rows, 16 x 8,192 cached, 64/8 heads of 128: 106 : 117; 64 rows, 131,072: 91 :
// 108; 32 rows, 16 x 4,096, 40/20: 119 : 141; 512 rows, 4 x 16,384, 64/8: 175 : 125;
// alike for 160 rows, 8 x 2,000, 40/8: 35 : 36, and 192 rows, 8 x 8,000, 24/8 of 64:
// 62 : 62.
int attn_tc_tile_rows(int R) { return R <= 128 ? 128 : 256; }

cudaError_t prepare_attn_tc(bool bf16, int D) {
  cudaError_t e;
  if (D == 128) {
    e = bf16 ? prepare<true, 128, 1>() : prepare<false, 128, 1>();
    if (e == cudaSuccess) e = bf16 ? prepare<true, 128, 2>() : prepare<false, 128, 2>();
  } else {
    e = bf16 ? prepare<true, 64, 1>() : prepare<false, 64, 1>();
    if (e == cudaSuccess) e = bf16 ? prepare<true, 64, 2>() : prepare<false, 64, 2>();
  }
  return e;
}

cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int D, const void* kmap, const void* vmap,
                           cudaStream_t st) {
  const bool one = attn_tc_tile_rows(p.R) == 128;
  if (D == 128) {
    if (bf16) return one ? launch<true, 128, 1>(p, kmap, vmap, st) : launch<true, 128, 2>(p, kmap, vmap, st);
    return one ? launch<false, 128, 1>(p, kmap, vmap, st) : launch<false, 128, 2>(p, kmap, vmap, st);
  }
  if (bf16) return one ? launch<true, 64, 1>(p, kmap, vmap, st) : launch<true, 64, 2>(p, kmap, vmap, st);
  return one ? launch<false, 64, 1>(p, kmap, vmap, st) : launch<false, 64, 2>(p, kmap, vmap, st);
}

}  // namespace qmm
