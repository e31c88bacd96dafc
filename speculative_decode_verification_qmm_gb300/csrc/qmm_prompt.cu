// qmm_prompt.cu -- causal attention of a prompt's rows over the paged cache
// (qmm_prompt_attention in include/qmm.h), on the tcgen05 tensor cores.
//
// Mathematics.  Row i of a sequence with L earlier rows sees the cache's rows j <= L + i.
// One pass over them with a running softmax, as in qmm_attn_tc.cu:
//   S = Q K^T;  P = 2^(c S - m), l += P;  O += P V;  out = O / l
// S, O and the statistics in fp32, P rounded to 16 bits for its product; m may lag
// behind the row's maximum by up to 8, O is rescaled when it grows more.
//
// Work.  A row tile is as many whole tokens of one key/value head's g query heads
// as fit into 128 NQ rows, and reads the cache tiles (128 rows) up to its last
// token's.  All (sequence, head, row tile, cache tile) units of the call are cut into
// equal contiguous ranges, one a CTA: long and short prompts, and few rows behind a
// long prefix, load the SMs alike.  Because a row tile's number of cache tiles grows with
// its place, the units before it are a sum of ceil((L + k i) / 128), which has a
// closed form by Euclid's algorithm (floor_sum).  What is cut leaves (O, m, l)
// partials to qmm_attn_join.cu.
//   warps 0 .. 4 NQ - 1   softmax, rescaling, output; a thread owns a row
//   two warps (NQ = 2: one) issue the MMAs
//   two warps             load K and V, tensor copies of 16 rows, a ring each; Q by both
// With NQ = 2 the row tiles take turns: O += P V of one, then its next S, while the
// other's softmax runs.
//
// Later rows than a row's own must not count, whatever they hold.  Their scores
// are replaced; of V, where 0 times NaN would, the loading warp takes the values that
// are not finite out of the tiles that some row of the item does not see wholly, and
// the rows that see them add them at the end.
// Every wait is bounded; on a timeout the CTA records it, its roles run out of
// their loops without waiting, copies and MMAs in flight are drained and tensor
// memory is freed.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "qmm_attn.cuh"
#include "qmm_attn.h"
#include "qmm_prompt.cuh"
#include "qmm_tc.cuh"

namespace qmm {

namespace {

constexpr int TK = 128;      // cache rows of a tile
constexpr int BAD_BUFS = 16; // more than twice the segments that the rings hold
constexpr int BAD_WORDS = 8; // an item's tokens after its first: at most 255
constexpr int ITEM_WEIGHT = 3;

// Two MMA warps and two loading warps beside four softmax warps; with two row tiles an MMA
// warp and three loading warps beside eight.
constexpr int threads_of(int NQ) { return NQ == 1 ? 256 : 384; }
// Registers a thread with two row tiles: what three groups of four warps are launched with, and
// what the two softmax groups and the third one go on with.
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 216, REGS_OTHER = 72;
static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * REGS_LAUNCH, "registers of a CTA");

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
  // kfull[KS], kempty[KS], vfull[VS], vempty[VS], vland[VS], qfull, qempty, sfull[2],
  // sfree[2], pfull[4], odone, olast[2], oempty[2], drain
  static constexpr int NBAR = 2 * KS + 3 * VS + 16;
  static constexpr int BAD = BAR + NBAR * 8;        // rows with non-finite V, by segment
  static constexpr int FLAG = BAD + BAD_BUFS * BAD_WORDS * 4;  // [0] abort, [1] tensor memory
  static constexpr int START = FLAG + 16;           // the CTA's share, and the cursor at its start
  static constexpr int BYTES = START + 48;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// Operands in shared memory with 128-byte swizzle, as in qmm_attn_tc.cu: the upper
// word of a descriptor is the same for all, a step along K adds to the lower one.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

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

// ---------------------------------------------------------------- division of the work
// sum of floor((a i + b) / m) over i < n <= 2^24, by Euclid's algorithm; m at most 128, b below 2^32.
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += ((int64_t)n * (n - 1) >> 1) * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += (int64_t)n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;  // below 128 * 2^24 + 128
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Cache tiles of the first `count` row tiles of a sequence with L earlier and n new rows.
__device__ __forceinline__ int64_t units_before(int L, int n, int per, int count) {
  const int full = n / per < count ? n / per : count;
  int64_t u = floor_sum((uint32_t)full, TK, (uint32_t)per, (uint32_t)L + per + TK - 1);
  if (count > full) u += ((int64_t)L + n + TK - 1) / TK;
  return u;
}

// Earlier rows L, new rows n of sequence b and the first of them; none where the
// table, or the call's rows, cannot hold them.
__device__ __forceinline__ bool prompt_sizes(const PromptParams& p, int b, int& L, int& n, int& first) {
  L = __ldg(p.a.lens + b);
  first = __ldg(p.starts + b);
  const int end = __ldg(p.starts + b + 1);
  const bool ok = L >= 0 && first >= 0 && end >= first && end <= p.N &&
                  (int64_t)L + (end - first) <= (int64_t)p.a.table_width << p.a.page_shift;
  n = ok ? end - first : 0;
  if (!ok) L = first = 0;
  return ok;
}

// A place in the call's work: an item (sequence, head, row tile) weighs its cache tiles
// and ITEM_WEIGHT more, which lie before the first tile, for what it costs to begin and
// end.
struct Cursor {
  int b, h, rt;
  int w;               // weight of the item that lies before the place
  int tiles;           // cache tiles of the item
  int L, n, first;     // of the sequence
};

__device__ __forceinline__ int64_t weight_before(const PromptParams& p, int L, int n, int count) {
  return units_before(L, n, p.per, count) + (int64_t)ITEM_WEIGHT * count;
}

__device__ __forceinline__ int tiles_of(const PromptParams& p, const Cursor& c) {
  const int end = (c.rt + 1) * p.per;
  return (c.L + (end < c.n ? end : c.n) + TK - 1) / TK;
}

// The start of CTA c's share of the work, and the share's weight, for every lane of a warp.
__device__ __forceinline__ Cursor begin(const PromptParams& p, int lane, int c, int64_t& left) {
  int64_t W = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    int64_t w = 0;
    if (b0 + lane < p.a.B) {
      int L, n, first;
      if (!prompt_sizes(p, b0 + lane, L, n, first) && c == 0) atomicOr(p.a.status, DEV_ERR_INDEX);
      w = weight_before(p, L, n, (n + p.per - 1) / p.per) * p.a.Hkv;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
    W += w;
  }
  // no CTA without a share between two that have one: the joining kernel counts on it
  const int G = W < p.a.grid ? (int)W : p.a.grid;
  Cursor cur{};
  left = 0;
  if (c >= G) return cur;
  const int64_t u0 = W * c / G;
  left = W * (c + 1) / G - u0;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    int L = 0, n = 0, first = 0;
    int64_t w = 0;
    if (b0 + lane < p.a.B) {
      prompt_sizes(p, b0 + lane, L, n, first);
      w = weight_before(p, L, n, (n + p.per - 1) / p.per) * p.a.Hkv;
    }
    int64_t inc = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, before + inc > u0);
    if (past) {
      const int who = __ffs(past) - 1;
      cur.b = b0 + who;
      cur.L = __shfl_sync(0xFFFFFFFFu, L, who);
      cur.n = __shfl_sync(0xFFFFFFFFu, n, who);
      cur.first = __shfl_sync(0xFFFFFFFFu, first, who);
      before += __shfl_sync(0xFFFFFFFFu, inc - w, who);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  const int all = (cur.n + p.per - 1) / p.per;
  const int64_t a_head = weight_before(p, cur.L, cur.n, all);
  const int64_t rem = u0 - before;
  cur.h = (int)(rem / a_head);
  const int64_t in_head = rem - cur.h * a_head;
  // the last row tile that begins at or before the place, 32 candidates at a time
  int lo = 0, hi = all;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool le = at < hi && weight_before(p, cur.L, cur.n, at) <= in_head;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, le));
    lo += k * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  cur.rt = lo;
  cur.w = (int)(in_head - weight_before(p, cur.L, cur.n, lo));
  cur.tiles = tiles_of(p, cur);
  return cur;
}

// Takes what the share has of the cursor's item: its cache tiles from `tile` on, and how
// many.  The cursor moves behind them.
__device__ __forceinline__ int take(Cursor& c, int64_t& left, int& tile) {
  const int64_t rest = c.tiles + ITEM_WEIGHT - c.w;
  const int w = rest < left ? (int)rest : (int)left;
  tile = c.w > ITEM_WEIGHT ? c.w - ITEM_WEIGHT : 0;
  c.w += w;
  left -= w;
  return c.w > ITEM_WEIGHT ? c.w - ITEM_WEIGHT - tile : 0;
}

// On to the next item.
__device__ __forceinline__ void next(const PromptParams& p, Cursor& c) {
  c.w = 0;
  if ((int64_t)++c.rt * p.per >= c.n) {
    c.rt = 0;
    if (++c.h == p.a.Hkv) {
      c.h = 0;
      do {
        if (++c.b >= p.a.B) return;
        prompt_sizes(p, c.b, c.L, c.n, c.first);
      } while (c.n == 0);
    }
  }
  c.tiles = tiles_of(p, c);
}

// Rows r0 .. left - 1 of a V tile without what is not finite (each row that has some is told
// to `found`), and zeros in the rows from `left` on, by a warp.
template <bool BF16, int D, typename F>
__device__ __forceinline__ void clean(uint32_t tile, int r0, int left, int lane, F found) {
  constexpr int CH = D / 8, HALF = TK * 128, BATCH = 8;
  const int ch = lane % CH, end = left * CH;
  auto place = [&](int id) {
    const int row = id / CH;
    return tile + (ch >> 3) * HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
  };
  auto put = [](uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  };
  for (int id = r0 * CH + lane; id < end; id += 32 * BATCH) {
    uint4 v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (id + 32 * i < end) v[i] = lds128(place(id + 32 * i));
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (id + 32 * i < end && any_nonfinite<BF16>(v[i])) {
        put(place(id + 32 * i), make_uint4(zero_nonfinite<BF16>(v[i].x), zero_nonfinite<BF16>(v[i].y),
                                           zero_nonfinite<BF16>(v[i].z), zero_nonfinite<BF16>(v[i].w)));
        found((id + 32 * i) / CH);
      }
  }
  for (int id = (left > 0 ? left : 0) * CH + lane; id < TK * CH; id += 32) put(place(id), make_uint4(0u, 0u, 0u, 0u));
}

template <bool BF16, int D, int NQ>
__global__ void __launch_bounds__(threads_of(NQ), 1)
    prompt_kernel(const __grid_constant__ PromptParams pp, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D, NQ>;
  const AttnParams& p = pp.a;
  constexpr int ROWS = NQ * 128;
  constexpr int SUB = NQ, SW = TK / SUB;  // steps that P is handed over in, columns of one
  constexpr int NB = 2 / NQ;              // buffers of S of a row tile
  constexpr uint32_t IDESC_S = tc_idesc_n(BF16 ? 1u : 0u, TK);
  constexpr uint32_t IDESC_O = tc_idesc_n(BF16 ? 1u : 0u, D) | (1u << 16);  // B along N
  // tensor memory columns: NB times S, then O, of each row tile
  constexpr uint32_t COL_O = NB * TK;
  constexpr uint32_t COL_Q = 256;  // of the second row tile
  constexpr int MMA_WARP = NQ * 4, MMA_WARPS = 2 / NQ, LOAD_WARP = MMA_WARP + MMA_WARPS;
  constexpr int Q_WARP = NQ == 2 ? LOAD_WARP + 2 : -1;  // (NQ = 1: both loading warps)
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t b_kfull = base + S::BAR, b_kempty = b_kfull + S::KS * 8, b_vfull = b_kempty + S::KS * 8,
                 b_vempty = b_vfull + S::VS * 8, b_vland = b_vempty + S::VS * 8, b_qfull = b_vland + S::VS * 8,
                 b_qempty = b_qfull + 8, b_sfull = b_qempty + 8, b_sfree = b_sfull + 16, b_pfull = b_sfree + 16,
                 b_odone = b_pfull + 32, b_olast = b_odone + 8, b_oempty = b_olast + 16, b_drain = b_oempty + 16;
  // sfull, sfree: [row tile], NQ = 1: [buffer]; pfull: [row tile][step], NQ = 1: [buffer]
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + S::FLAG);
  unsigned* s_bad = reinterpret_cast<unsigned*>(smem + S::BAD);

  if (tid == 0) {
    for (int i = 0; i < S::KS; ++i) {
      mbar_init(b_kfull + 8 * i, 1);
      mbar_init(b_kempty + 8 * i, 1);
    }
    for (int i = 0; i < S::VS; ++i) {
      mbar_init(b_vfull + 8 * i, 1);
      mbar_init(b_vempty + 8 * i, 1);
      mbar_init(b_vland + 8 * i, 1);
    }
    mbar_init(b_qfull, NQ == 1 ? 2 : 1);
    mbar_init(b_qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_sfree + 8 * i, 1);
      mbar_init(b_olast + 8 * i, 1);
      mbar_init(b_oempty + 8 * i, 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(b_pfull + 8 * i, 4);
    mbar_init(b_odone, 1);
    mbar_init(b_drain, MMA_WARPS);
    for (int i = 0; i < BAD_BUFS * BAD_WORDS; ++i) s_bad[i] = 0;
    s_flag[0] = 0;
    if (base & 1023u) {
      atomicOr(p.status, DEV_ERR_SMEM_ALIGN);
      s_flag[0] = 1;
    }
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(base + S::FLAG + 4, 512);
  // What the call reads is there, and the last call's partials were read; only
  // then may the joining kernel take its place.
  pdl_wait();
  pdl_trigger();
  int64_t share;
  Cursor cur;
  if (warp == 0) {
    cur = begin(pp, lane, blockIdx.x, share);
    if (lane == 0) {
      *reinterpret_cast<int64_t*>(smem + S::START) = share;
      *reinterpret_cast<Cursor*>(smem + S::START + 8) = cur;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  share = *reinterpret_cast<const int64_t*>(smem + S::START);
  cur = *reinterpret_cast<const Cursor*>(smem + S::START + 8);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, (uint32_t)s_flag[1], 0);

  if (tid == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  const uint64_t lim = p.wait_limit_ns;
  auto fail = [&](int code) {
    if (!s_flag[0]) atomicOr(p.status, code);
    s_flag[0] = 1;
  };
  // Tokens and rows of the cursor's row tile.
  auto tokens = [&] {
    const int left = cur.n - cur.rt * pp.per;
    return left < pp.per ? left : pp.per;
  };

  // Rows of Q, by threads `id` of `STEP` CH; rows past the item's stay as they are, and so do
  // their results.
  auto load_q = [&](int id, auto step) {
    constexpr int CH = D / 8, STEP = decltype(step)::value / CH;  // 16-byte chunks of a row, rows at a time
    const int rows = tokens() * p.g, ch = id % CH;
    const int dt = STEP / p.g, dh = STEP % p.g;
    int row = id / CH, t = row / p.g, h = row % p.g;
    const uint16_t* src = p.q + (int64_t)(cur.first + cur.rt * pp.per) * p.q_st + (int64_t)cur.h * p.g * p.q_sh + ch * 8;
#pragma unroll 8
    for (; row < rows; row += STEP) {
      cp_async16(base + S::Q + (row >> 7) * S::TILE + (ch >> 3) * S::HALF + (row & 127) * 128 +
                     (((ch & 7) ^ (row & 7)) << 4),
                 src + t * p.q_st + h * p.q_sh, 16);
      t += dt, h += dh;
      if (h >= p.g) h -= p.g, ++t;
    }
    cp_async_commit();
    cp_async_wait<0>();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b_qfull);
  };

  if (warp >= MMA_WARP) {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
  if (warp >= LOAD_WARP) {
    // ------------------------------------------------------------ load
    const bool is_v = warp > LOAD_WARP;
    const uint32_t full = is_v ? b_vfull : b_kfull, empty = is_v ? b_vempty : b_kempty;
    const uint32_t ring = base + (is_v ? S::V : S::K);
    const int slots = is_v ? S::VS : S::KS;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    constexpr int BLOCKS = TK / 16;  // 16 rows, one tensor copy a half
    bool ok = s_flag[0] == 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xFFFFFFFFu, ok && wait_or_abort(bar, parity, lim, s_flag));
      if (!ok && lane == 0) fail(DEV_ERR_TIMEOUT_EMPTY);
    };
    int slot = 0, round = 0, seg = 0;
    unsigned landing = 0, landed = 0;  // bits by slot: a copy counts on vland; vland's parity
    while (share > 0 && ok) {
      int tile;
      const int count = take(cur, share, tile);
      if (count > 0) {
        if (NQ == 1 || warp == Q_WARP) {
          if (seg > 0) wait(b_qempty, (uint32_t)((seg - 1) & 1));
          if (!ok) break;
          if constexpr (NQ == 1)
            load_q((warp - LOAD_WARP) * 32 + lane, std::integral_constant<int, 64>());
          else
            load_q(lane, std::integral_constant<int, 32>());
        }
        ++seg;
      }
      // Lane i < BLOCKS looks up the page of the tile's block i, a tile ahead.  An
      // id out of range is reported; rows of page 0 take its place.
      const int first_token = cur.rt * pp.per;
      const int end = cur.L + first_token + tokens();  // rows that a row of the item sees
      const int all_see = cur.L + first_token;         // the last row that every one sees
      int ahead = 0;
      auto lookup = [&](int j) {
        const int jb = j * TK + lane * 16;
        ahead = 0;
        if (lane < BLOCKS && jb < end) {
          ahead = __ldg(p.table + cur.b * p.ld_table + (jb >> p.page_shift));
          if (ahead < 0 || ahead >= p.n_pages) {
            atomicOr(p.status, DEV_ERR_INDEX);
            ahead = 0;
          }
        }
      };
      const int copies = NQ == 2 && warp == Q_WARP ? 0 : count;
      if (copies > 0) lookup(tile);
      for (int j = 0; j < copies; ++j) {
        const int j0 = (tile + j) * TK;
        const int pid = ahead;
        if (j + 1 < count) lookup(tile + j + 1);
        if (round > 0) wait(empty + 8 * slot, (uint32_t)((round - 1) & 1));
        if (!ok) break;
        const int left = end - j0 < TK ? end - j0 : TK;  // rows of the tile that count
        const int blocks = (left + 15) / 16;
        const bool masked = is_v && j0 + TK - 1 > all_see;
        const uint32_t bar = (masked ? b_vland : full) + 8 * slot, dst = ring + slot * S::TILE;
        landing = masked ? landing | 1u << slot : landing & ~(1u << slot);
        if (lane == 0) mbar_arrive_expect_tx(bar, blocks * 16 * D * 2);
        __syncwarp();
        if (lane < blocks) {
          const int64_t row = p.row0 + (((int64_t)pid * p.Hkv + cur.h) << p.page_shift) +
                              ((j0 + lane * 16) & ((1 << p.page_shift) - 1));
#pragma unroll
          for (int half = 0; half < D / 64; ++half)
            tma_load_2d(dst + half * S::HALF + lane * 2048, map, half * 64, (int)row, bar);
        }
        if (masked) {
          wait(bar, landed >> slot & 1u);
          if (!ok) {  // (the copy is waited for below, with this slot's round counted)
            if (++slot == slots) slot = 0, ++round;
            break;
          }
          landed ^= 1u << slot;
          landing &= ~(1u << slot);
          clean<BF16, D>(dst, all_see + 1 > j0 ? all_see + 1 - j0 : 0, left, lane, [&](int row) {
            const int k = j0 + row - all_see - 1;
            atomicOr(s_bad + ((seg - 1) & (BAD_BUFS - 1)) * BAD_WORDS + (k >> 5), 1u << (k & 31));
          });
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + 8 * slot);
        }
        if (++slot == slots) slot = 0, ++round;
      }
      if (share > 0) next(pp, cur);
    }
    cp_async_wait<0>();
    // Tensor copies in flight land before the CTA leaves: the last tile of every
    // slot.  Always: another role can give up after this one's last look at the flag.
    for (int i = 0; i < slots; ++i) {
      const int rounds = i < slot ? round + 1 : round;
      if (rounds > 0 && lane == 0) {
        const bool on_land = landing >> i & 1u;
        if (!mbar_wait_bounded(on_land ? b_vland + 8 * i : full + 8 * i, on_land ? landed >> i & 1u : (rounds - 1) & 1,
                               1000000000ull))
          atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else {
    // ------------------------------------------------------------ MMA issue
    // The warp stays together and one elected lane issues (see qmm_attn_tc.cu).
    uint32_t leader;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
    const int who = warp - MMA_WARP;  // NQ = 1: 0 Q K^T, 1 P V
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
    // O of row tile q += a step's P (at column a) times its rows of the V tile in `slot`
    auto product_o = [&](int q, int slot, int sub, uint32_t a, bool first) {
      const uint32_t d = tmem + q * COL_Q + COL_O;
      const uint32_t b = desc_lo_mn(base + S::V + slot * S::TILE + sub * SW * 128, S::HALF);
      tc_fence_after();
      if (leader) {
        mma_ts(d, a, b, IDESC_O, !first);
#pragma unroll
        for (int kk = 1; kk < SW / 16; ++kk) mma_ts(d, a + kk * 8, b + kk * (2048 >> 4), IDESC_O, 1);
      }
    };
    int n = 0, seg = 0;         // tiles and segments so far (parities, and whether there was one)
    int slot = 0, round = 0;    // of the tile of K or V
    int vslot = 0, vround = 0;  // of the tile of V, where one warp issues both
    while (share > 0 && ok) {
      int tile;
      const int count = take(cur, share, tile);
      if (count == 0) {  // (a share can end before an item's first tile)
        if (share > 0) next(pp, cur);
        continue;
      }
      if constexpr (NQ == 2) {
        // O += P V of a row tile, then S of its next cache tile, then the other row tile
        for (int j = -1; j < count && ok; ++j) {
          if (j < 0 && !need(b_qfull, seg)) break;
          for (int q = 0; q < 2 && ok; ++q) {
            if (j >= 0) {
              if (q == 0 && !need(b_vfull + 8 * vslot, vround)) break;
              if (j == 0 && seg > 0 && !need(b_oempty + 8 * q, seg - 1)) break;
#pragma unroll
              for (int sub = 0; sub < SUB; ++sub) {
                if (!need(b_pfull + 8 * (2 * q + sub), n)) break;
                product_o(q, vslot, sub, tmem + q * COL_Q + sub * (SW / 2), j == 0 && sub == 0);
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
              if (leader) tc_commit(b_sfull + 8 * q);
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
          product_o(0, slot, 0, tmem + (n & 1) * TK, j == 0);
          if (leader) tc_commit(b_odone);
          if (leader) tc_commit(b_sfree + 8 * (n & 1));
          if (leader && j + 1 == count) tc_commit(b_olast);
          if (leader) tc_commit(b_vempty + 8 * slot);
          if (++slot == S::VS) slot = 0, ++round;
        }
      }
      ++seg;
      if (share > 0) next(pp, cur);
    }
    // all MMAs of the CTA have ended before tensor memory is given back
    if (leader) {
      tc_commit(b_drain);
      if (!mbar_wait_bounded(b_drain, 0, 1000000000ull)) atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    // a thread holds a row's 128 scores: registers of the other warps go to these
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int q = warp >> 2;
    const int row = q * 128 + (warp & 3) * 32 + lane;
    const int t_in = row / p.g, i_row = row - t_in * p.g;  // token in the row tile, query head
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
    while (share > 0) {
      int tile;
      const int count = take(cur, share, tile);
      if (count == 0) {
        if (share > 0) next(pp, cur);
        continue;
      }
      const int toks = tokens();
      const bool in = t_in < toks, idle = !__any_sync(0xFFFFFFFFu, in);
      const int t_row = cur.rt * pp.per + t_in;
      const int all_see = cur.L + cur.rt * pp.per;
      const int sees = cur.L + t_row;  // the last row that this one sees
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < count; ++j) {
        const int n = done + j;
        const uint32_t t_s = tl + (NB == 2 ? (n & 1) * TK : 0);
        const uint32_t pfull = b_pfull + 8 * (NQ == 2 ? 2 * q : n & 1);
        need(b_sfull + 8 * (NQ == 2 ? q : n & 1), NQ == 2 ? n : n >> 1);
        if (!ok) continue;
        if (idle) {  // no row of the warp is the item's: whatever P is, nobody looks
          if (lane == 0)
            for (int sub = 0; sub < SUB; ++sub) mbar_arrive(pfull + 8 * sub);
          continue;
        }
        tc_fence_after();
        const int j0 = (tile + j) * TK;
        uint32_t v[TK / 32][32];  // the row's scores
#pragma unroll
        for (int c = 0; c < TK / 32; ++c) tmem_ld32(t_s + c * 32, v[c]);
        tmem_wait_ld();
        if (j0 + TK - 1 > all_see) {
          const int last = sees - j0;
#pragma unroll
          for (int c = 0; c < TK / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i > last) v[c][i] = 0xFF800000u;  // -inf
        }
        float mx;
        {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < TK / 32; ++c)
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
            // NQ = 2: this S was computed after the last product with V had ended
            if (NQ == 1 && !need(b_odone, n - 1)) continue;
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
        for (int c = 0; c < TK / 32; ++c) {
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
          if ((c + 1) % (SW / 32) == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + 8 * (c / (SW / 32)));
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }

      // ------------------------------------------------ end of the segment
      need(b_olast + 8 * q, seg);
      tc_fence_after();
      const bool last_tile = tile + count == cur.tiles, whole = tile == 0 && last_tile;
      if (tid == 0 && !last_tile)
        p.cuts[blockIdx.x] = make_int4(cur.first + cur.rt * pp.per, cur.h, toks * p.g, attn_cut(true, tile == 0));
      constexpr int PART = ROWS * (D + 2);
      float* part = p.ws + ((int64_t)blockIdx.x * 2 + (tile == 0 ? 1 : 0)) * PART;
      const unsigned* bad = s_bad + (seg & (BAD_BUFS - 1)) * BAD_WORDS;
      unsigned any_bad = 0;
#pragma unroll
      for (int i = 0; i < BAD_WORDS; ++i) any_bad |= bad[i];
      // read by all, not yet written again
      if (tid < BAD_WORDS) s_bad[((seg + BAD_BUFS / 2) & (BAD_BUFS - 1)) * BAD_WORDS + tid] = 0;
      const int64_t at = cur.first + t_row;  // the row in q, out and lse
      const float inv = in && l != 0.f ? 1.f / l : 0.f;
      uint16_t* const to16 = p.out + at * p.o_st + (int64_t)(cur.h * p.g + i_row) * p.o_sh;
      if (whole && !any_bad && !idle) {
        // The rows' outputs are taken out of tensor memory, which is then free for the
        // next item, before they are stored.
        uint32_t w[D / 2];
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          tmem_ld32(t_o + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            w[(c + i) / 2] = pack16<BF16>(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_oempty + 8 * q);
        // Four lanes exchange their rows' 32 columns, so that they store a row's 64 bytes at a time.
        uint16_t* rows[4];
        bool have[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rows[k] = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)to16, (lane & 28) + k)) + (lane & 3) * 8;
          have[k] = __shfl_sync(0xFFFFFFFFu, in && ok, (lane & 28) + k);
        }
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t* x = w + c / 2;
#pragma unroll
          for (int h = 2; h > 0; h >>= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!(k & h))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t &lo = x[k * 4 + e], &hi = x[(k | h) * 4 + e];
                  const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, lane & h ? lo : hi, h);
                  (lane & h ? lo : hi) = y;
                }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (have[k])
              *reinterpret_cast<uint4*>(rows[k] + c) = make_uint4(x[k * 4], x[k * 4 + 1], x[k * 4 + 2], x[k * 4 + 3]);
        }
        if (ok && in && p.lse) p.lse[at * p.Hq + cur.h * p.g + i_row] = (m + log2f(l)) * 0.69314718055994531f;
        done += count;
        ++seg;
        if (share > 0) next(pp, cur);
        continue;
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(t_o + c, v);
        tmem_wait_ld();
        float a[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(v[i]);
        if (any_bad && in) {
          // the non-finite values of V, for the rows that see them
          const uint16_t* qr = p.q + at * p.q_st + (int64_t)(cur.h * p.g + i_row) * p.q_sh;
          for (int k = 0; k < 32 * BAD_WORDS && all_see + 1 + k <= sees; ++k) {
            if (!(bad[k >> 5] >> (k & 31) & 1u)) continue;
            const int r = all_see + 1 + k;
            int id = __ldg(p.table + cur.b * p.ld_table + (r >> p.page_shift));
            if (id < 0 || id >= p.n_pages) id = 0;
            const int64_t where = id * p.page_stride + ((int64_t)cur.h << p.page_shift) * D +
                                  (int64_t)(r & ((1 << p.page_shift) - 1)) * D;
            float s = 0.f;
            for (int d = 0; d < D; ++d) s = fmaf(unpack16<BF16>(qr[d]), unpack16<BF16>(p.k_pool[where + d]), s);
            const float w = ex2(fmaf(s, p.scale_log2, -(m == -INFINITY ? 0.f : m)));
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = unpack16<BF16>(p.v_pool[where + c + i]);
              if (!isfinite(x)) a[i] += w * x;
            }
          }
        }
        if (!ok || idle) continue;
        if (whole) {
          if (in) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(to16 + c + k) = make_uint4(
                  pack16<BF16>(a[k] * inv, a[k + 1] * inv), pack16<BF16>(a[k + 2] * inv, a[k + 3] * inv),
                  pack16<BF16>(a[k + 4] * inv, a[k + 5] * inv), pack16<BF16>(a[k + 6] * inv, a[k + 7] * inv));
          }
          continue;
        }
        // Eight lanes exchange their rows' 32 columns, so that they store a row at
        // a time, four columns each.
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
        float* to = part + (row & ~7) * D + c + (lane & 7) * 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(to + k * D) = make_float4(a[k * 4], a[k * 4 + 1], a[k * 4 + 2], a[k * 4 + 3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_oempty + 8 * q);
      if (whole) {
        if (ok && in && p.lse) p.lse[at * p.Hq + cur.h * p.g + i_row] = (m + log2f(l)) * 0.69314718055994531f;
      } else if (ok) {
        part[ROWS * D + row] = m;
        part[ROWS * D + ROWS + row] = l;
      }
      done += count;
      ++seg;
      if (share > 0) next(pp, cur);
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
  if (NQ == 2) {
    // a CTA launched with fewer registers than its groups ask for would wait for them
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, prompt_kernel<BF16, D, NQ>);
    if (e != cudaSuccess) return e;
    if (at.numRegs < REGS_LAUNCH) return cudaErrorInvalidKernelImage;
  }
  return cudaFuncSetAttribute(prompt_kernel<BF16, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, NQ>::BYTES);
}

template <bool BF16, int D, int NQ>
cudaError_t launch(const PromptParams& p, const void* kmap, const void* vmap, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.grid);
  cfg.blockDim = dim3(threads_of(NQ));
  cfg.dynamicSmemBytes = Smem<D, NQ>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_kernel<BF16, D, NQ>, p, *static_cast<const CUtensorMap*>(kmap),
                            *static_cast<const CUtensorMap*>(vmap));
}

template <bool BF16, int D>
cudaError_t launch_rows(const PromptParams& p, const void* kmap, const void* vmap, cudaStream_t st) {
  return p.rows == 128 ? launch<BF16, D, 1>(p, kmap, vmap, st) : launch<BF16, D, 2>(p, kmap, vmap, st);
}

}  // namespace

int prompt_tile_cache_rows() { return TK; }

cudaError_t prepare_prompt(bool bf16, int D) {
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

cudaError_t launch_prompt(const PromptParams& p, bool bf16, int D, const void* kmap, const void* vmap, cudaStream_t st) {
  if (D == 128) return bf16 ? launch_rows<true, 128>(p, kmap, vmap, st) : launch_rows<false, 128>(p, kmap, vmap, st);
  return bf16 ? launch_rows<true, 64>(p, kmap, vmap, st) : launch_rows<false, 64>(p, kmap, vmap, st);
}

}  // namespace qmm
