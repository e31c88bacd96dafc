// qmm_attn_tc.cu -- tree attention for more than 32 rows per key/value head, on
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
// behind the true maximum by up to 8 (P <= 256): O is rescaled, by the softmax
// warps and through their registers, only when a row of the warp grows more.
//   warps 0 .. 4 NQ - 1   softmax, rescaling, output (four warps a row tile)
//   warp 4 NQ             one thread issues the MMAs
//   the last three warps  load: cp.async of 32 KB tiles (D = 128) of K and V in
//                         turn into a ring, Q once a segment, the tree's nodes
//                         from the caller's rows (and on to the cache)
// Why this split.  At 128 rows a tile of K and V (64 KB) takes 1.5 us of an
// SM's share of the HBM stream, and its two products 0.55 us of the tensor cores
// and its 16,384 exponentials about as long: with one row tile the stream is the
// bound, and S is double-buffered so that Q K^T of the next tile runs under the
// softmax.  With two, each tile of K and V serves 256 rows, and the products of
// one row tile run under the softmax of the other.  Tensor memory: NQ = 1 holds
// S twice (256 columns) and O; NQ = 2 S and O for both (512).  P overwrites the
// first half of its S.
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
constexpr int LOAD_WARPS = 3;  // and the MMA warp: one warpgroup
constexpr int LAG = 3;    // groups of cp.async in flight behind the newest
constexpr int BAD_BUFS = 8;

template <int D, int NQ>
struct Smem {
  static constexpr int TILE = TK * D * 2;           // one of K, V; also 128 rows of Q
  static constexpr int HALF = TK * 128;             // 64 columns of a tile
  static constexpr int SLOTS = (D == 128 ? 7 - NQ : 10);
  static constexpr int Q = 0;
  static constexpr int RING = Q + NQ * TILE;
  static constexpr int BAR = RING + SLOTS * TILE;
  // full[SLOTS], empty[SLOTS], qfull, qempty, sfull[2], pfull[2], odone[2], oempty[2], drain
  static constexpr int NBAR = 2 * SLOTS + 11;
  static constexpr int BAD = BAR + NBAR * 8;        // nodes with non-finite V, by segment
  static constexpr int FLAG = BAD + BAD_BUFS * 8;   // [0] abort, [1] tensor memory, [2] last
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

template <int N>
__device__ __forceinline__ void bar_named(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
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
__global__ void __launch_bounds__(NQ * 128 + 128, 1) attn_tc_kernel(const __grid_constant__ AttnParams p) {
  using S = Smem<D, NQ>;
  constexpr int ROWS = NQ * 128;
  constexpr int SOFT = NQ * 128;  // softmax threads
  constexpr int SLOTS = S::SLOTS;
  constexpr uint32_t IDESC_S = tc_idesc_n(BF16 ? 1u : 0u, TK);
  constexpr uint32_t IDESC_O = tc_idesc_n(BF16 ? 1u : 0u, D) | (1u << 16);  // B along N
  // tensor memory columns: NQ = 1: S twice, O; NQ = 2: S, O of each row tile
  constexpr uint32_t COL_O = NQ == 1 ? 2 * TK : TK;
  constexpr uint32_t COL_Q = 256;  // of the second row tile
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t b_full = base + S::BAR, b_empty = b_full + SLOTS * 8, b_qfull = b_empty + SLOTS * 8,
                 b_qempty = b_qfull + 8, b_sfull = b_qempty + 8, b_pfull = b_sfull + 16, b_odone = b_pfull + 16,
                 b_oempty = b_odone + 16, b_drain = b_oempty + 16;
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + S::FLAG);
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(smem + S::BAD);

  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(b_full + 8 * i, LOAD_WARPS);
      mbar_init(b_empty + 8 * i, 1);
    }
    mbar_init(b_qfull, LOAD_WARPS);
    mbar_init(b_qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_pfull + 8 * i, 4);
      mbar_init(b_odone + 8 * i, 1);
      mbar_init(b_oempty + 8 * i, 4);
    }
    mbar_init(b_drain, 1);
    for (int i = 0; i < BAD_BUFS; ++i) s_bad[i] = 0;
    s_flag[0] = 0;
    if (base & 1023u) {
      atomicOr(p.status, DEV_ERR_SMEM_ALIGN);
      s_flag[0] = 1;
    }
    fence_mbar_init();
  }
  constexpr int MMA_WARP = NQ * 4;
  if (warp == MMA_WARP) tmem_alloc(base + S::FLAG + 4, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)s_flag[1];

  const uint64_t lim = p.wait_limit_ns;
  auto fail = [&](int code) {
    if (!s_flag[0]) atomicOr(p.status, code);
    s_flag[0] = 1;
  };
  int64_t W, u0, u1;
  int G;
  AttnCursor cur = attn_begin<TK>(p, lane, blockIdx.x, gridDim.x, W, G, u0, u1);
  const int64_t head = (int64_t)D << p.page_shift;
  if (warp > MMA_WARP) {
    // ------------------------------------------------------------ load
    const int lw = warp - (MMA_WARP + 1);
    constexpr int CH = D / 8;                     // 16-byte chunks of a row
    constexpr int PER = 16 * CH / 32;             // chunks of a block per lane
    // A tile is eight blocks of 16 rows, each in one page; warp lw takes blocks
    // lw, lw + LOAD_WARPS, ...
    constexpr int BLOCKS = TK / 16, MINE = (BLOCKS + LOAD_WARPS - 1) / LOAD_WARPS;
    bool ok = s_flag[0] == 0;
    uint32_t pend[LAG];  // barriers of the groups in flight, oldest first
    int pend_n = 0;
#pragma unroll
    for (int i = 0; i < LAG; ++i) pend[i] = 0;

    // The warp's blocks of a tile with nodes, once they have landed: on to the
    // cache, and non-finite V out of the product.
    auto finish = [&](const AttnCursor& c, uint32_t dst, int j0, int kind, int seg) {
      uint16_t* pool = kind == 1 ? p.k_pool : p.v_pool;
#pragma unroll 1
      for (int i = 0; i < MINE * PER; ++i) {
        const int blk = lw + i / PER * LOAD_WARPS, id = i % PER * 32 + lane;  // the chunks that it requested
        const int row = blk * 16 + id / CH, ch = id % CH;
        if (blk >= BLOCKS) break;
        const int j = j0 + row, t = j - c.L;
        if (t < 0 || t >= c.n) continue;
        const uint32_t so = dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        uint4 v = lds128(so);
        if (c.rt == 0) {
          const int pid = __ldg(p.table + c.b * p.ld_table + (j >> p.page_shift));
          if (pid >= 0 && pid < p.n_pages)
            *reinterpret_cast<uint4*>(pool + pid * p.page_stride + c.h * head +
                                      (int64_t)(j & ((1 << p.page_shift) - 1)) * D + ch * 8) = v;
          else
            atomicOr(p.status, DEV_ERR_INDEX);
        }
        if (kind == 2 && any_nonfinite<BF16>(v)) {
          v.x = zero_nonfinite<BF16>(v.x);
          v.y = zero_nonfinite<BF16>(v.y);
          v.z = zero_nonfinite<BF16>(v.z);
          v.w = zero_nonfinite<BF16>(v.w);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(so), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
          atomicOr(s_bad + (seg & (BAD_BUFS - 1)), 1ull << t);
        }
      }
    };
    auto hand_on = [&](uint32_t bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // One more group is under way: hand on the oldest once LAG are behind it.
    auto push = [&](uint32_t bar) {
      cp_async_commit();
      if (pend_n == LAG) {
        cp_async_wait<LAG>();
        hand_on(pend[0]);
#pragma unroll
        for (int i = 0; i + 1 < LAG; ++i) pend[i] = pend[i + 1];
        pend[LAG - 1] = bar;
      } else {
#pragma unroll
        for (int i = 0; i < LAG; ++i)
          if (i == pend_n) pend[i] = bar;
        ++pend_n;
      }
    };
    auto flush = [&]() {
      cp_async_wait<0>();
#pragma unroll
      for (int i = 0; i < LAG; ++i)
        if (i < pend_n) hand_on(pend[i]);
      pend_n = 0;
    };
    // Before a wait everything under way is handed on: what is waited for may
    // depend on it.
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (lim != 0 && __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
      flush();
      const bool got = __all_sync(0xFFFFFFFFu, wait_or_abort(bar, parity, lim, s_flag));
      if (!got && lane == 0) fail(DEV_ERR_TIMEOUT_EMPTY);
      return got;
    };
    int slot = 0, round = 0;  // of the next tile of K or V
    // The page ids of the warp's blocks of a cache tile.
    auto pages = [&](const AttnCursor& c, int j, int (&ids)[MINE]) {
#pragma unroll
      for (int x = 0; x < MINE; ++x) {
        const int blk = lw + x * LOAD_WARPS, jb = j * TK + blk * 16;
        ids[x] = blk < BLOCKS && jb < c.L ? __ldg(p.table + c.b * p.ld_table + (jb >> p.page_shift)) : 0;
      }
    };
    auto tile = [&](const AttnCursor& c, int j, int kind, int seg, const int (&ids)[MINE]) {
      if (ok && round > 0) ok = wait(b_empty + 8 * slot, (uint32_t)((round - 1) & 1));
      if (!ok) return;
      const uint32_t dst = base + S::RING + slot * S::TILE;
      const int j0 = j * TK;
      const uint16_t* pool = (kind == 1 ? p.k_pool : p.v_pool) + c.h * head;
      const uint16_t* fresh = kind == 1 ? p.kn + c.b * p.k_sb + c.h * p.k_sh : p.vn + c.b * p.v_sb + c.h * p.v_sh;
      const int64_t fresh_st = kind == 1 ? p.k_st : p.v_st;
      bool bad_page = false;
#pragma unroll
      for (int x = 0; x < MINE; ++x) {
        const int blk = lw + x * LOAD_WARPS;
        if (blk >= BLOCKS) break;
        const int jb = j0 + blk * 16;
        const bool valid = ids[x] >= 0 && ids[x] < p.n_pages;
        bad_page |= !valid;
        const uint32_t have = valid ? 16 : 0;
        const uint16_t* from = pool + (valid ? ids[x] : 0) * p.page_stride +
                               (int64_t)(jb & ((1 << p.page_shift) - 1)) * D;
        if (jb + 16 <= c.L) {
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int id = i * 32 + lane, row = blk * 16 + id / CH, ch = id % CH;
            cp_async16(dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4), from + id * 8, have);
          }
        } else {
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int id = i * 32 + lane, row = blk * 16 + id / CH, ch = id % CH;
            const int t = j0 + row - c.L;
            const bool node = t >= 0 && t < c.n;
            const uint32_t bytes = node ? 16 : (t < 0 ? have : 0);
            const uint16_t* src = node ? fresh + t * fresh_st + ch * 8 : (bytes ? from + id * 8 : p.k_pool);
            cp_async16(dst + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4), src, bytes);
          }
        }
      }
      if (bad_page) atomicOr(p.status, DEV_ERR_INDEX);
      if (j0 + TK > c.L && j0 < c.L + c.n) {
        cp_async_commit();
        flush();
        finish(c, dst, j0, kind, seg);
        hand_on(b_full + 8 * slot);
      } else {
        push(b_full + 8 * slot);
      }
      if (++slot == SLOTS) slot = 0, ++round;
    };

    int seg = 0;
    for (int64_t u = u0; u < u1 && ok; ++seg) {
      int64_t left = cur.ntiles - cur.tile;
      if (left > u1 - u) left = u1 - u;
      const int first = cur.tile, count = (int)left;
      if (seg > 0) ok = wait(b_qempty, (uint32_t)((seg - 1) & 1));
      if (!ok) break;
      for (int id = lw * 32 + lane; id < ROWS * CH; id += LOAD_WARPS * 32) {
        const int row = id / CH, ch = id % CH;  // row of all NQ tiles
        const int r = cur.rt * ROWS + row, t = r / p.g, h = r - t * p.g;
        const uint16_t* src = p.q + cur.b * p.q_sb + t * p.q_st + (int64_t)(cur.h * p.g + h) * p.q_sh + ch * 8;
        cp_async16(base + S::Q + (row >> 7) * S::TILE + (ch >> 3) * S::HALF + (row & 127) * 128 +
                       (((ch & 7) ^ (row & 7)) << 4),
                   r < p.R ? src : p.q, r < p.R ? 16 : 0);
      }
      push(b_qfull);
      // in the order in which the MMAs read them; page ids are fetched a tile ahead
      int ids[MINE] = {}, ahead[MINE], old[MINE];
      pages(cur, first, ahead);
      for (int j = 0; j < count; ++j) {
#pragma unroll
        for (int x = 0; x < MINE; ++x) old[x] = ids[x], ids[x] = ahead[x];
        if (j + 1 < count) pages(cur, first + j + 1, ahead);
        tile(cur, first + j, 1, seg, ids);
        if constexpr (NQ == 1) {
          if (j > 0) tile(cur, first + j - 1, 2, seg, old);
        } else {
          tile(cur, first + j, 2, seg, ids);
        }
      }
      if constexpr (NQ == 1) tile(cur, first + count - 1, 2, seg, ids);
      cur.tile = first + count - 1;
      attn_next<TK>(p, cur);
      u += count;
    }
    flush();
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      bool ok = s_flag[0] == 0;
      auto need = [&](uint32_t bar, int phase) {
        if (ok && !wait_or_abort(bar, (uint32_t)(phase & 1), lim, s_flag)) {
          fail(DEV_ERR_TIMEOUT_FULL);
          ok = false;
        }
        return ok;
      };
      int slot = 0, round = 0;  // of the next tile of K or V
      auto next = [&]() {
        if (++slot == SLOTS) slot = 0, ++round;
      };
      int done = 0;  // cache tiles whose Q K^T was issued before this segment (parities only)
      auto qk = [&](int q, int buf, int sl) {
        const uint32_t a = desc_lo(base + S::Q + q * S::TILE), b = desc_lo(base + S::RING + sl * S::TILE);
        const uint32_t d = tmem + q * COL_Q + buf * TK;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr uint32_t STEP = 32 >> 4, HALF = S::HALF >> 4;
          const uint32_t o = (uint32_t)(kk >> 2) * HALF + (uint32_t)(kk & 3) * STEP;
          mma_ss(d, a + o, b + o, IDESC_S, kk > 0);
        }
        tc_commit(b_sfull + 8 * (NQ == 1 ? buf : q));
      };
      auto pv = [&](int q, int buf, int sl, bool first) {
        const uint32_t a = tmem + q * COL_Q + buf * TK, d = tmem + q * COL_Q + COL_O;
        const uint32_t b = desc_lo_mn(base + S::RING + sl * S::TILE, S::HALF);
        tc_fence_after();
        mma_ts(d, a, b, IDESC_O, !first);
#pragma unroll
        for (int kk = 1; kk < TK / 16; ++kk) mma_ts(d, a + kk * 8, b + kk * (2048 >> 4), IDESC_O, 1);
        tc_commit(b_odone + 8 * q);
      };
      int seg = 0;
      for (int64_t u = u0; u < u1 && ok; ++seg) {
        int64_t left = cur.ntiles - cur.tile;
        if (left > u1 - u) left = u1 - u;
        const int count = (int)left;
        if (!need(b_qfull, seg)) break;
        if constexpr (NQ == 1) {
          for (int j = 0; j <= count && ok; ++j) {
            if (j < count) {
              const int n = done + j;
              if (!need(b_full + 8 * slot, round)) break;
              // its S holds P of two tiles ago until that product is done (at a
              // segment's start the product of the last tile is the newest one)
              if (j == 0 ? n >= 1 && !need(b_odone, n - 1) : n >= 2 && !need(b_odone, n - 2)) break;
              qk(0, n & 1, slot);
              tc_commit(b_empty + 8 * slot);
              if (j == count - 1) tc_commit(b_qempty);
              next();
            }
            if (j > 0) {
              const int n = done + j - 1;
              if (!need(b_full + 8 * slot, round)) break;
              if (!need(b_pfull + 8 * (n & 1), n >> 1)) break;
              if (j == 1 && seg > 0 && !need(b_oempty, seg - 1)) break;
              pv(0, n & 1, slot, j == 1);
              tc_commit(b_empty + 8 * slot);
              next();
            }
          }
        } else {
          if (!need(b_full + 8 * slot, round)) break;
          for (int q = 0; q < 2 && ok; ++q)
            if (done == 0 || need(b_odone + 8 * q, done - 1)) qk(q, 0, slot);
          if (!ok) break;
          tc_commit(b_empty + 8 * slot);
          if (count == 1) tc_commit(b_qempty);
          next();
          for (int j = 0; j < count && ok; ++j) {
            const int n = done + j;
            const bool more = j + 1 < count;
            if (!need(b_full + 8 * slot, round)) break;
            const int vslot = slot;
            next();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (!need(b_pfull + 8 * q, n)) break;
              if (j == 0 && seg > 0 && !need(b_oempty + 8 * q, seg - 1)) break;
              pv(q, 0, vslot, j == 0);
              if (q == 1) tc_commit(b_empty + 8 * vslot);
              if (more) {
                if (q == 0 && !need(b_full + 8 * slot, round)) break;
                // P lies in S: the next S may follow when its product is done
                if (!need(b_odone + 8 * q, n)) break;
                qk(q, 0, slot);
              }
            }
            if (!ok) break;
            if (more) {
              tc_commit(b_empty + 8 * slot);
              if (j + 2 == count) tc_commit(b_qempty);
              next();
            }
          }
        }
        done += count;
        cur.tile += count - 1;
        attn_next<TK>(p, cur);
        u += count;
      }
      // all MMAs of the CTA have ended before tensor memory is given back
      tc_commit(b_drain);
      if (!mbar_wait_bounded(b_drain, 0, 1000000000ull)) atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + q * COL_Q;
    const uint32_t t_o = tl + COL_O;
    bool ok = s_flag[0] == 0;
    auto need = [&](uint32_t bar, int64_t phase) {
      if (ok) {
        const bool got = __all_sync(0xFFFFFFFFu, wait_or_abort(bar, (uint32_t)(phase & 1), lim, s_flag));
        if (!got) {
          if (lane == 0) fail(DEV_ERR_TIMEOUT_FULL);
          ok = false;
        }
      }
      return ok;
    };
    int64_t done = 0;
    int seg = 0;
    for (int64_t u = u0; u < u1; ++seg) {
      int64_t left = cur.ntiles - cur.tile;
      if (left > u1 - u) left = u1 - u;
      const int count = (int)left;
      const int r = cur.rt * ROWS + q * 128 + row;
      const bool in = r < p.R;
      const uint64_t bits = in ? attn_bits(p, cur.b, cur.n, r) : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < count; ++j) {
        const int64_t n = done + j;
        const int buf = NQ == 1 ? (int)(n & 1) : 0;
        const uint32_t t_s = tl + buf * TK;
        if (!need(b_sfull + 8 * (NQ == 1 ? buf : q), NQ == 1 ? n >> 1 : n)) continue;
        tc_fence_after();
        const int t0 = (cur.tile + j) * TK - cur.L;  // node of the tile's first row, if it is one
        const bool edge = t0 + TK > 0;
        // One row tile: the row's 128 scores stay in registers.  Two: 64 at a time
        // (168 registers a thread), the second half first, as P of the first
        // half then takes the place of scores that are in registers.
        constexpr int PARTS = NQ, CPP = TK / 32 / PARTS;
        uint32_t v[CPP][32];
        auto fetch = [&](int part) {
#pragma unroll
          for (int c = 0; c < CPP; ++c) tmem_ld32(t_s + (part * CPP + c) * 32, v[c]);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int c = 0; c < CPP; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int t = t0 + (part * CPP + c) * 32 + i;
                if (t >= 0 && (t >= 64 || !(bits >> t & 1))) v[c][i] = 0xFF800000u;  // -inf
              }
          }
        };
        float mx = -INFINITY;
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) {
          fetch(part);
          float x[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < CPP; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              x[(i >> 1) & 3] = fmaxf(x[(i >> 1) & 3], fmaxf(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])));
          mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        }
        mx *= p.scale_log2;
        if (__any_sync(0xFFFFFFFFu, mx > m + 8.f)) {
          const float mn = fmaxf(m, mx);
          const float a = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= a;
          if (j > 0) {
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
        for (int part = 0; part < PARTS; ++part) {
          if (part > 0) fetch(part);
#pragma unroll
          for (int c = 0; c < CPP; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float2 e = fma2(make_float2(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), c2, m2);
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], e);
              w[i / 2] = pack16<BF16>(e.x, e.y);
            }
            tmem_st16(t_s + (part * CPP + c) * 16, w);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        // Every product is waited for in turn, before the one that follows it can
        // start: a parity tells one phase of a barrier from the next, no more.
        if (n > 0 && !need(b_odone + 8 * q, n - 1)) continue;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_pfull + 8 * (NQ == 1 ? buf : q));
      }

      // ------------------------------------------------ end of the segment
      need(b_odone + 8 * q, done + count - 1);
      tc_fence_after();
      const int64_t item_u = u - cur.tile;  // the item's first unit
      const bool last_tile = cur.tile + count == cur.ntiles;
      const bool whole = cur.tile == 0 && last_tile;
      constexpr int PART = ROWS * (D + 2);
      float* part = p.ws + ((int64_t)blockIdx.x * 2 + (item_u >= u0 ? 1 : 0)) * PART;
      const int t_row = r / p.g, i_row = r - t_row * p.g;
      const bool live = in && t_row < cur.n;
      const unsigned long long bad = s_bad[seg & (BAD_BUFS - 1)];
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
        if (!ok) continue;
        if (whole) {
          if (in) write16(t_row, i_row, c, a, inv);
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(part + (q * 128 + row) * D + c + i) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_oempty + 8 * q);
      if (whole) {
        if (ok && in && p.lse)
          p.lse[((int64_t)cur.b * p.T + t_row) * p.Hq + cur.h * p.g + i_row] =
              live ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        bar_named<SOFT>(1);
      } else {
        if (ok) {
          part[ROWS * D + q * 128 + row] = m;
          part[ROWS * D + ROWS + q * 128 + row] = l;
        }
        __threadfence();
        bar_named<SOFT>(1);
        const int c0 = attn_owner(item_u, W, G), c1 = attn_owner(item_u + cur.ntiles - 1, W, G);
        if (tid == 0) {
          int is_last = 0;
          if (s_flag[0] == 0) {
            is_last = atomicAdd(p.counters + c0, 1) == c1 - c0;
            if (is_last) p.counters[c0] = 0;
          }
          s_flag[2] = is_last;
        }
        bar_named<SOFT>(1);
        if (s_flag[2]) {
          __threadfence();
          attn_join<BF16, D, ROWS, SOFT / 32>(p, cur, c0, c1, warp, lane);
        }
        bar_named<SOFT>(1);
      }
      if (tid == 0) s_bad[seg & (BAD_BUFS - 1)] = 0;
      done += count;
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
cudaError_t launch(const AttnParams& p, int ctas, cudaStream_t st) {
  attn_tc_kernel<BF16, D, NQ><<<(unsigned)ctas, NQ * 128 + 128, Smem<D, NQ>::BYTES, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

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

cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int D, int ctas, cudaStream_t st) {
  const bool one = attn_tc_tile_rows(p.R) == 128;
  if (D == 128) {
    if (bf16) return one ? launch<true, 128, 1>(p, ctas, st) : launch<true, 128, 2>(p, ctas, st);
    return one ? launch<false, 128, 1>(p, ctas, st) : launch<false, 128, 2>(p, ctas, st);
  }
  if (bf16) return one ? launch<true, 64, 1>(p, ctas, st) : launch<true, 64, 2>(p, ctas, st);
  return one ? launch<false, 64, 1>(p, ctas, st) : launch<false, 64, 2>(p, ctas, st);
}

}  // namespace qmm
