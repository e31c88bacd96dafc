// qmm_prompt.cu -- causal attention of a prompt's rows over the paged cache
// (qmm_prompt_attention in include/qmm.h), on the tcgen05 tensor cores.
//
// Mathematics.  Row i of a sequence with L earlier rows sees the cache's rows j <= L + i.
// One pass over them with a running softmax, as in qmm_attn_tc.cu:
//   S = Q K^T;  P = 2^(c S - m), l += P;  O += P V;  out = O / l
// S, O and the statistics in fp32, P rounded to 16 bits for its product, which takes operands
// of one type (V's; a second product for what the rounding leaves would take as long again); l is
// the sum of the unrounded P.  m may lag behind the row's maximum by up to 8, O is rescaled when
// it grows more.
//
// Work.  A row tile is as many whole tokens of one key/value head's g query heads
// as fit into 128 NQ rows, and reads the cache tiles (128 rows) up to its last
// token's.  All (sequence, head, row tile, cache tile) units of the call are cut into
// equal contiguous ranges, one a CTA: long and short prompts, and few rows behind a
// long prefix, load the SMs alike.  Because a row tile's number of cache tiles grows with
// its place, the units before it are a sum of ceil((L + k i) / 128), which has a
// closed form by Euclid's algorithm (floor_sum).  What is cut leaves (O, m, l)
// partials to qmm_attn_join.cu.
//   warps 0 .. 7          softmax, rescaling, output; a thread owns a row, or, NQ = 1, half of
//                         its columns: then its two threads tell each other their maxima
//   two warps (NQ = 2: one) issue the MMAs
//   two warps             load K and V, tensor copies of 16 rows, a ring each; Q by both
// With NQ = 2 the row tiles take turns: O += P V of one, then its next S, while the
// other's softmax runs.
//
// Later rows than a row's own must not count, whatever they hold.  Their scores
// are replaced; of V, where 0 times NaN would, the loading warp takes the values that
// are not finite out of the tiles that some row of the item does not see wholly, and
// the rows that see them add them at the end.
// What bounds it.  Heads of 128: the tensor cores with shared memory, which delivers both operands
// of S at its full rate while TMA writes; 8,192 rows of 40/20 heads 507 us, 1,360 TFLOP/s, 72 % of a large
// product's rate; 512 rows behind 65,536, 64/8 heads, 746 us, 1,480 TFLOP/s.  Heads of 64: the softmax,
// whose exponentials take as long as the products and cannot all run beside them; 512 rows behind
// 16,384, 64/8 heads, 152 us, 921 TFLOP/s.  Short prompts: an item's start and end, and the joining launch.
// Tried and slower: waits by test instead of try (2 to 3 %), the wait for P's place after the first 32
// exponentials instead of before them (heads of 64: 4 %), a register split between roles (spills stay).
//
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
// What an item costs besides its tiles, in tiles.  (1, 3, 6 and 12, us: 9 ragged prompts of up to
// 1,501 rows, 28/4 heads of 64: 114, 112, 116, 126; 2,048 rows, 32/4 heads of 128: 72, 59, 60, 66; 16 of up
// to 300, 64/8: 68, 66, 68, 66.)
constexpr int ITEM_WEIGHT = 3;

// Threads of a row: a single row tile's softmax has nothing else to run beside it.  (One : two, us: 75
// rows, 40/20 heads of 128, 10.0 : 9.6; 8 times 300, 64/8, 57 : 49; 16 times 200 behind 500, 12/12, 42.1 : 39.8;
// 1,024, 32/4 heads of 64, 24.3 : 23.4; most others within 2 %.  Two row tiles with two, heads of 64: 9
// ragged prompts 113 : 119, 512 behind 20,000 98 : 102.)
template <int NQ>
constexpr int SPLIT = NQ == 1 ? 2 : 1;
// Four softmax warps a row tile and thread of a row, two MMA warps, two loading warps.
template <int NQ>
constexpr int THREADS = NQ * 128 * SPLIT<NQ> + 128;
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
  // kfull[KS], kempty[KS], vfull[VS], vempty[VS], vland[VS], sfull[2], sfree[2],
  // pfull[4], odone[2], olast[2], oempty[2], qfull, qempty, drain, met[8]
  static constexpr int NBAR = 2 * KS + 3 * VS + 25;
  static constexpr int BAD = BAR + NBAR * 8;        // rows with non-finite V, by segment
  static constexpr int FLAG = BAD + BAD_BUFS * BAD_WORDS * 4;  // [0] abort, [1] tensor memory
  static constexpr int START = FLAG + 16;           // the CTA's share, and the places of its first and last unit
  static constexpr int MEET = START + 80;           // what a row's threads tell each other: [turn][thread][row]
  static constexpr int BYTES = MEET + (SPLIT<NQ> > 1 ? 2 * 2 * NQ * 128 * 4 : 0);
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

// A warp's bounded wait for a phase of a barrier; it gives up too when another role did.  All
// branches are the warp's, not a lane's: with loops of single lanes and an error path of
// one lane behind them, a pair of cache tiles took 2,950 cycles in a model of the kernel
// below, and takes 2,490.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t lim, volatile int* flag) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  const long long limit = (long long)(lim < (1ull << 40) ? lim : (1ull << 40)) * 2;
  while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xFFFFFFFFu, *flag || clock64() - t0 > limit)) return false;
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

// The same for m = TK and a power of two.
__device__ __forceinline__ int64_t floor_sum_pow2(uint32_t n, uint32_t a, uint32_t b) {
  if (a >= TK) return ((int64_t)n * (n - 1) >> 1) * (a / TK) + (int64_t)n * (b / TK);
  const int sa = 31 - __clz(a), sk = 31 - __clz(TK / a);
  auto steps = [&](uint32_t x) {  // sum of floor(i a / TK) over i < x
    const int64_t q = x >> sk;
    return (q * (q - 1) >> 1 << sk) + q * (x & ((1u << sk) - 1));
  };
  const uint32_t c = b >> sa;
  return steps(n + c) - steps(c);
}

// Cache tiles of the first `count` row tiles of a sequence with L earlier and n new rows.
__device__ __forceinline__ int64_t units_before(int L, int n, int per, int count) {
  const bool pow2 = (per & (per - 1)) == 0;
  const int most = pow2 ? n >> (31 - __clz(per)) : n / per, full = most < count ? most : count;
  const uint32_t b = (uint32_t)L + per + TK - 1;
  int64_t u = pow2 ? floor_sum_pow2((uint32_t)full, (uint32_t)per, b) : floor_sum((uint32_t)full, TK, (uint32_t)per, b);
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

// Quotients of whole numbers that mostly fit into 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The place of the first (or last) unit of CTA c's share of the work, and the share's weight,
// for every lane of a warp.
__device__ __forceinline__ Cursor begin(const PromptParams& p, int lane, int c, bool last, int64_t& share) {
  Cursor cur{};
  int64_t W = 0, head = 0;  // of a key/value head of the lane's sequence
  auto look = [&](int b0) {
    cur.L = cur.n = cur.first = 0;
    bool ok = true;
    if (b0 + lane < p.a.B) ok = prompt_sizes(p, b0 + lane, cur.L, cur.n, cur.first);
    head = weight_before(p, cur.L, cur.n, (cur.n + p.per - 1) / p.per);
    return ok;
  };
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    if (!look(b0) && c == 0 && !last) atomicOr(p.a.status, DEV_ERR_INDEX);
    int64_t w = head * p.a.Hkv;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
    W += w;
  }
  // no CTA without a share between two that have one: the joining kernel counts on it
  const int G = W < p.a.grid ? (int)W : p.a.grid;
  share = 0;
  if (c >= G) return cur;
  const int64_t first = quotient(W * c, G), end = quotient(W * (c + 1), G), u0 = last ? end - 1 : first;
  share = end - first;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    if (p.a.B > 32) look(b0);
    const int64_t w = head * p.a.Hkv;
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
      cur.L = __shfl_sync(0xFFFFFFFFu, cur.L, who);
      cur.n = __shfl_sync(0xFFFFFFFFu, cur.n, who);
      cur.first = __shfl_sync(0xFFFFFFFFu, cur.first, who);
      head = __shfl_sync(0xFFFFFFFFu, head, who);
      before += __shfl_sync(0xFFFFFFFFu, inc - w, who);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  const int64_t rem = u0 - before;
  cur.h = (int)quotient(rem, head);
  const int64_t in_head = rem - cur.h * head;
  // the last row tile that begins at or before the place, 32 candidates at a time
  int lo = 0, hi = (cur.n + p.per - 1) / p.per;
  int64_t at_lo = 0;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const int64_t w = weight_before(p, cur.L, cur.n, at < hi ? at : hi);
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && w <= in_head));
    if (k > 0) at_lo = __shfl_sync(0xFFFFFFFFu, w, k - 1);
    lo += k * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  cur.rt = lo;
  cur.w = (int)(in_head - at_lo);
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

// On to the next item.  (Sequences without rows are passed one by one: 16 prompts of 100 behind 500, 32/4
// heads of 128, 35 us alone, 41 spread over 256 sequences, 71 over 1,024, 206 over 4,096.)
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
// to `found`), and zeros in the rows from `left` on, by a warp.  (Batches whose branch is
// the warp's: with one for each chunk a tile's 128 rows took 10,000 cycles.)
template <bool BF16, int D, typename F>
__device__ __forceinline__ void clean(uint32_t tile, int r0, int left, int lane, F found) {
  constexpr int CH = D / 8, HALF = TK * 128, BATCH = 8, ROWS = 32 * BATCH / CH;  // rows of a batch
  const int ch = lane % CH;
  auto place = [&](int row) { return tile + (ch >> 3) * HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4); };
  auto put = [](uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  };
  int row = r0 + lane / CH;
  for (int first = r0; first < left; first += ROWS, row += ROWS) {
    uint4 v[BATCH];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      // (past the end the last row again)
      v[i] = lds128(place(row + i * (32 / CH) < left ? row + i * (32 / CH) : left - 1));
      bad |= any_nonfinite<BF16>(v[i]);
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll 1
      for (int i = 0; i < BATCH; ++i) {
        const int r = row + i * (32 / CH);
        if (r >= left) break;
        const uint4 x = lds128(place(r));
        if (!any_nonfinite<BF16>(x)) continue;
        put(place(r), make_uint4(zero_nonfinite<BF16>(x.x), zero_nonfinite<BF16>(x.y), zero_nonfinite<BF16>(x.z),
                                 zero_nonfinite<BF16>(x.w)));
        found(r);
      }
      __syncwarp();
    }
  }
  for (int r = left + lane / CH; r < TK; r += 32 / CH) put(place(r), make_uint4(0u, 0u, 0u, 0u));
}

template <bool BF16, int D, int NQ>
__global__ void __launch_bounds__(THREADS<NQ>, 1)
    prompt_kernel(const __grid_constant__ PromptParams pp, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D, NQ>;
  const AttnParams& p = pp.a;
  constexpr int ROWS = NQ * 128;
  constexpr int H = SPLIT<NQ>, W = TK / H;  // columns of S of a thread
  // Steps that P is handed over in, columns of one.  Two threads of a row: one, since either may
  // still rescale its part of O.
  constexpr int SUB = H == 2 ? 1 : 2, SW = TK / SUB;
  constexpr int NB = 2 / NQ;              // buffers of S of a row tile
  constexpr uint32_t IDESC_S = tc_idesc_n(BF16 ? 1u : 0u, TK);
  constexpr uint32_t IDESC_O = tc_idesc_n(BF16 ? 1u : 0u, D) | (1u << 16);  // B along N
  // tensor memory columns: NB times S, then O, of each row tile
  constexpr uint32_t COL_O = NB * TK;
  constexpr uint32_t COL_Q = D == 128 ? 256 : 192;  // of the second row tile
  // With two row tiles P lies where its S did, or, heads of 64, in columns of its own: then
  // the next S need not wait for the product of P and V, but for the softmax to have read S.
  constexpr bool APART = NQ == 2 && D == 64;
  constexpr uint32_t COL_P = 384;  // APART, 64 columns a row tile
  // NQ = 1: one warp issues all Q K^T, the other all P V.  APART: each issues both for its row
  // tile.  Else one issues everything (the commits of two would wait behind each other's
  // products), and the other loads Q.
  constexpr bool ONE = NQ == 2 && !APART;
  constexpr int ISSUERS = APART ? 2 : 1;  // that use a tile of K, or of V
  constexpr int MMA_WARP = NQ * 4 * H, MMA_WARPS = 2, LOAD_WARP = MMA_WARP + MMA_WARPS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  // (constant distances from base: nothing to keep in registers)
  constexpr uint32_t O_KFULL = S::BAR, O_KEMPTY = O_KFULL + S::KS * 8, O_VFULL = O_KEMPTY + S::KS * 8,
                     O_VEMPTY = O_VFULL + S::VS * 8, O_VLAND = O_VEMPTY + S::VS * 8, O_SFULL = O_VLAND + S::VS * 8,
                     O_SFREE = O_SFULL + 16, O_PFULL = O_SFREE + 16, O_ODONE = O_PFULL + 32, O_OLAST = O_ODONE + 16,
                     O_OEMPTY = O_OLAST + 16, O_QFULL = O_OEMPTY + 16, O_QEMPTY = O_QFULL + 8, O_DRAIN = O_QEMPTY + 8, O_MET = O_DRAIN + 8;
  // sfull, sfree: [row tile], NQ = 1: [buffer]; pfull: [row tile][step], NQ = 1: [buffer][step];
  // met: [row tile][warp's rows]
  volatile int* s_flag = reinterpret_cast<volatile int*>(smem + S::FLAG);
  unsigned* s_bad = reinterpret_cast<unsigned*>(smem + S::BAD);

  if (tid == 0) {
    for (int i = 0; i < S::KS; ++i) {
      mbar_init(base + O_KFULL + 8 * i, 1);
      mbar_init(base + O_KEMPTY + 8 * i, ISSUERS);
    }
    for (int i = 0; i < S::VS; ++i) {
      mbar_init(base + O_VFULL + 8 * i, 1);
      mbar_init(base + O_VEMPTY + 8 * i, ISSUERS);
      mbar_init(base + O_VLAND + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(base + O_SFULL + 8 * i, 1);
      mbar_init(base + O_SFREE + 8 * i, APART ? 4 * H : 1);
      mbar_init(base + O_ODONE + 8 * i, 1);
      mbar_init(base + O_OLAST + 8 * i, 1);
      mbar_init(base + O_OEMPTY + 8 * i, 4 * H);
    }
    for (int i = 0; i < 4; ++i) mbar_init(base + O_PFULL + 8 * i, 4 * H);
    mbar_init(base + O_QFULL, 1);
    mbar_init(base + O_QEMPTY, 1);
    mbar_init(base + O_DRAIN, MMA_WARPS);
    for (int i = 0; i < 8; ++i) mbar_init(base + O_MET + 8 * i, 2);
    for (int i = 0; i < BAD_BUFS * BAD_WORDS; ++i) s_bad[i] = 0;
    // a limit of 0 makes every wait give up
    s_flag[0] = base & 1023u ? DEV_ERR_SMEM_ALIGN : (p.wait_limit_ns == 0 ? DEV_ERR_TIMEOUT_EMPTY : 0);
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(base + S::FLAG + 4, 512);
  // What the call reads is there, and the last call's partials were read; only
  // then may the joining kernel take its place.
  pdl_wait();
  pdl_trigger();
  if (warp < 2) {
    int64_t share;
    const Cursor c = begin(pp, lane, blockIdx.x, warp == 1, share);
    if (lane == 0) {
      *reinterpret_cast<Cursor*>(smem + S::START + 8 + 32 * warp) = c;
      if (warp == 0) *reinterpret_cast<int64_t*>(smem + S::START) = share;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (tid == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  const uint64_t lim = p.wait_limit_ns;
  auto fail = [&](int code) { s_flag[0] = code; };  // by all lanes of a warp
  // The share's parts, each a place and a weight; every role reads them anew, for registers
  // of its own.  What the CTA has of its last item, if others go on with it, comes first:
  // then the CTAs that a long cache's items are spread over read about the same rows at a time, and
  // these once from memory.  (512 rows behind 65,536, 64/8 heads of 128: 4.3 GB in order.)
  auto start = [&](int part, Cursor& c) -> int64_t {
    const int64_t share = *reinterpret_cast<const int64_t*>(smem + S::START);
    const Cursor* at = reinterpret_cast<const Cursor*>(smem + S::START + 8);
    c = at[0];
    if (share == 0) return 0;
    const int64_t in_last = at[1].w + 1;  // of the share, if the last item begins in it
    const bool split = in_last < share && in_last < at[1].tiles + ITEM_WEIGHT;
    if (part == 0 && split) {
      c = at[1];
      c.w = 0;
      return in_last;
    }
    return split ? share - in_last : (part == 0 ? share : 0);
  };
  // On to the next item of the share.
  auto go_on = [&](Cursor& c, int64_t& share, int& part) {
    if (share > 0)
      next(pp, c);
    else
      share = part == 0 ? start(++part, c) : 0;
    return share > 0;
  };
  // Tokens of the cursor's row tile.
  auto tokens = [&](const Cursor& c) {
    const int left = c.n - c.rt * pp.per;
    return left < pp.per ? left : pp.per;
  };

  if (warp >= LOAD_WARP) {
    // ------------------------------------------------------------ load
    Cursor cur;
    int part = 0;
    int64_t share = start(part, cur);
    const bool is_v = warp > LOAD_WARP;
    const uint32_t full = base + (is_v ? O_VFULL : O_KFULL), empty = base + (is_v ? O_VEMPTY : O_KEMPTY);
    const uint32_t ring = base + (is_v ? S::V : S::K);
    const int slots = is_v ? S::VS : S::KS;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    constexpr int BLOCKS = TK / 16;  // 16 rows, one tensor copy a half
    bool ok = s_flag[0] == 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok && !warp_wait(bar, parity, lim, s_flag)) {
        fail(DEV_ERR_TIMEOUT_EMPTY);
        ok = false;
      }
    };
    int slot = 0, round = 0, seg = 0;
    unsigned landing = 0, landed = 0;  // bits by slot: a copy counts on vland; vland's parity
    for (bool on = share > 0; on && ok; on = go_on(cur, share, part)) {
      int tile;
      const int count = take(cur, share, tile);
      if (count > 0) ++seg;
      // Lane i < BLOCKS looks up the page of the tile's block i, a tile ahead.  An
      // id out of range is reported; rows of page 0 take its place.
      const int first_token = cur.rt * pp.per;
      const int end = cur.L + first_token + tokens(cur);  // rows that a row of the item sees
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
      if (count > 0) lookup(tile);
      for (int j = 0; j < count; ++j) {
        const int j0 = (tile + j) * TK;
        const int pid = ahead;
        if (j + 1 < count) lookup(tile + j + 1);
        if (round > 0) wait(empty + 8 * slot, (uint32_t)((round - 1) & 1));
        if (!ok) break;
        const int left = end - j0 < TK ? end - j0 : TK;  // rows of the tile that count
        const int blocks = (left + 15) / 16;
        const bool masked = is_v && j0 + TK - 1 > all_see;
        const uint32_t bar = (masked ? base + O_VLAND : full) + 8 * slot, dst = ring + slot * S::TILE;
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
    }
    // Tensor copies in flight land before the CTA leaves: the last tile of every
    // slot.  Always: another role can give up after this one's last look at the flag.
    for (int i = 0; i < slots; ++i) {
      const int rounds = i < slot ? round + 1 : round;
      if (rounds > 0 && lane == 0) {
        const bool on_land = landing >> i & 1u;
        if (!mbar_wait_bounded(on_land ? base + O_VLAND + 8 * i : full + 8 * i, on_land ? landed >> i & 1u : (rounds - 1) & 1,
                               1000000000ull))
          atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
      }
    }
  } else if (warp >= MMA_WARP) {
    // ------------------------------------------------------------ MMA issue
    // The warp stays together and one elected lane issues (see qmm_attn_tc.cu).
    uint32_t leader;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
    Cursor cur_next;
    int part = 0;
    int64_t share = start(part, cur_next);
    // What the products' operands come from is made uniform: they then live in uniform
    // registers.
    auto uniform = [](uint32_t x) { return __reduce_max_sync(0xFFFFFFFFu, x); };
    const uint32_t tmem = uniform((uint32_t)s_flag[1]);
    const int who = (int)uniform((uint32_t)(warp - MMA_WARP));
    bool ok = s_flag[0] == 0;
    auto need = [&](uint32_t bar, int phase) {
      if (!warp_wait(bar, (uint32_t)(phase & 1), lim, s_flag)) {
        fail(DEV_ERR_TIMEOUT_FULL);
        ok = false;
      }
      return ok;
    };
    // Requests row tile q's rows of Q of the item at c; rows past the item's stay as they are,
    // and so do their results.
    auto request_q = [&](int q, const Cursor& c) {
      constexpr int CH = D / 8, STEP = 32 / CH;  // 16-byte chunks of a row, rows at a time
      const int left = tokens(c) * p.g - q * 128, rows = left < 128 ? left : 128, ch = lane % CH;
      const int dt = STEP / p.g, dh = STEP % p.g;
      int row = lane / CH, t = (q * 128 + row) / p.g, h = (q * 128 + row) % p.g;
      const uint16_t* src = p.q + (int64_t)(c.first + c.rt * pp.per) * p.q_st + (int64_t)c.h * p.g * p.q_sh + ch * 8;
#pragma unroll 4
      for (; row < rows; row += STEP) {
        cp_async16(base + S::Q + q * S::TILE + (ch >> 3) * S::HALF + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   src + t * p.q_st + h * p.q_sh, 16);
        t += dt, h += dh;
        if (h >= p.g) h -= p.g, ++t;
      }
      cp_async_commit();
    };
    auto q_landed = [&] {
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
    };
    int n = 0, seg = 0;         // tiles and segments so far (parities, and whether there was one)
    int slot = 0, round = 0;    // of the tile of K
    int vslot = 0, vround = 0;  // of the tile of V
    // Barriers and columns of row tile q and tile n
    auto s_index = [&](int q, int n) { return (uint32_t)(NQ == 2 ? q : n & 1); };
    auto s_phase = [&](int n) { return NQ == 2 ? n : n >> 1; };
    auto s_column = [&](int q, int n) { return tmem + (NQ == 2 ? q * COL_Q : (n & 1) * TK); };
    // The segments one after the other; the next one is looked up ahead, for its Q.
    int count = 0, count_next = 0;
    bool on = share > 0, fresh = true;
    auto look_ahead = [&] {
      count_next = 0;
      while (on && count_next == 0) {  // (a part can end before an item's first tile)
        int from;
        if (!fresh && !(on = go_on(cur_next, share, part))) break;
        fresh = false;
        count_next = take(cur_next, share, from);
      }
      count_next = (int)uniform((uint32_t)count_next);
    };
    // S of row tile q and the segment's cache tile j, the call's n-th; `takes` and `leaves`: is
    // the first, the last to use the tile of K
    auto issue_s = [&](int q, int j, int n, bool takes, bool leaves) {
      if (ONE && j == 0 && takes && !need(base + O_QFULL, seg)) return false;
      if (!ONE && j == 0) q_landed();
      if (takes && !need(base + O_KFULL + 8 * slot, round)) return false;
      // S goes where S, or P, of the last tile but NB lies: until that one was read (APART), or
      // its product with V has ended
      if (n >= NB && !need(base + O_SFREE + 8 * s_index(q, n), s_phase(n) - 1)) return false;
      // (operands are worked out before the branch on the lane: in it, each would go to a
      // uniform register for every product anew, three times as slow)
      const uint32_t a = desc_lo(base + S::Q + q * S::TILE), b = desc_lo(base + S::K + slot * S::TILE), d = s_column(q, n);
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (uint32_t)(kk >> 2) * (S::HALF >> 4) + (uint32_t)(kk & 3) * (32 >> 4);
          mma_ss(d, a + o, b + o, IDESC_S, kk > 0);
        }
      }
      if (leader) tc_commit(base + O_SFULL + 8 * s_index(q, n));
      if (leader && leaves) tc_commit(base + O_KEMPTY + 8 * slot);
      if (leader && ONE && leaves && j + 1 == count) tc_commit(base + O_QEMPTY);
      if (leaves && ++slot == S::KS) slot = 0, ++round;
      if (!ONE && j + 1 == count && count_next > 0) {  // Q makes way for the next one
        if (!need(base + O_SFULL + 8 * s_index(q, n), s_phase(n))) return false;
        request_q(q, cur_next);
      }
      return true;
    };
    // O of row tile q += P times V, in the steps that P comes in
    auto issue_o = [&](int q, int j, int n, bool takes, bool leaves) {
      if (takes && !need(base + O_VFULL + 8 * vslot, vround)) return false;
      if (j == 0 && seg > 0 && !need(base + O_OEMPTY + 8 * q, seg - 1)) return false;
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        if (!need(base + O_PFULL + 8 * (2 * s_index(q, n) + sub), s_phase(n))) return false;
        const uint32_t a = (APART ? tmem + COL_P + q * 64 : s_column(q, n)) + sub * (SW / 2), d = tmem + q * COL_Q + COL_O;
        const uint32_t b = desc_lo_mn(base + S::V + vslot * S::TILE + sub * SW * 128, S::HALF);
        tc_fence_after();
        if (leader) {
          mma_ts(d, a, b, IDESC_O, sub > 0 || j > 0);
#pragma unroll
          for (int kk = 1; kk < SW / 16; ++kk) mma_ts(d, a + kk * 8, b + kk * (2048 >> 4), IDESC_O, 1);
        }
      }
      if (!ONE && leader) tc_commit(base + O_ODONE + 8 * q);
      if (!APART && leader) tc_commit(base + O_SFREE + 8 * s_index(q, n));
      if (leader && j + 1 == count) tc_commit(base + O_OLAST + 8 * q);
      if (leader && leaves) tc_commit(base + O_VEMPTY + 8 * vslot);
      if (leaves && ++vslot == S::VS) vslot = 0, ++vround;
      return true;
    };
    look_ahead();
    if (!ONE && (NQ == 2 || who == 0) && count_next > 0) request_q(who, cur_next);
    while (count_next > 0 && ok) {
      count = count_next;
      if constexpr (ONE) {
        if (who == 0) {
          // P V of a row tile, S of its next cache tile, then the other row tile
          if (!issue_s(0, 0, n, true, false) || !issue_s(1, 0, n, false, true)) break;
          for (int j = 0; j < count; ++j, ++n) {
            if (!issue_o(0, j, n, true, false)) break;
            if (j + 1 < count && !issue_s(0, j + 1, n + 1, true, false)) break;
            if (!issue_o(1, j, n, false, true)) break;
            if (j + 1 < count && !issue_s(1, j + 1, n + 1, false, true)) break;
          }
        } else {
          // Q, when the products with the last one have ended
          if (seg > 0 && !need(base + O_QEMPTY, seg - 1)) break;
          for (int q = 0; q < 2; ++q) request_q(q, cur_next);
          q_landed();
          if (lane == 0) mbar_arrive(base + O_QFULL);
        }
        look_ahead();
      } else {
        look_ahead();
        if constexpr (NQ == 1) {
          for (int j = 0; j < count && ok; ++j, ++n)
            if (who == 0)
              issue_s(0, j, n, true, true);
            else
              issue_o(0, j, n, true, true);
        } else if (issue_s(who, 0, n, true, true)) {
          // the next S first: its place is free long before P is there
          for (int j = 0; j < count; ++j, ++n) {
            if (j + 1 < count && !issue_s(who, j + 1, n + 1, true, true)) break;
            if (!issue_o(who, j, n, true, true)) break;
          }
        }
      }
      ++seg;
    }
    cp_async_wait<0>();
    // all MMAs of the CTA have ended before tensor memory is given back
    if (leader) {
      tc_commit(base + O_DRAIN);
      if (!mbar_wait_bounded(base + O_DRAIN, 0, 1000000000ull)) atomicOr(p.status, DEV_ERR_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ softmax
    Cursor cur;
    int part = 0;
    int64_t share = start(part, cur);
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, (uint32_t)s_flag[1], 0);
    const int q = warp / (4 * H), half = H == 2 ? warp >> 2 & 1 : 0;  // the row's thread
    const int row = q * 128 + (warp & 3) * 32 + lane;
    const int t_in = row / p.g, i_row = row - t_in * p.g;  // token in the row tile, query head
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + q * COL_Q;
    const uint32_t t_o = tl + COL_O;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    bool ok = s_flag[0] == 0;
    auto need = [&](uint32_t bar, int phase) {
      if (ok && !warp_wait(bar, (uint32_t)(phase & 1), lim, s_flag)) {
        fail(DEV_ERR_TIMEOUT_FULL);
        ok = false;
      }
      return ok;
    };
    // The row's threads give each other a value: f(one's own, the other's).
    float* const s_meet = reinterpret_cast<float*>(smem + S::MEET);
    const uint32_t met = base + O_MET + 8 * (q * 4 + (warp & 3));
    int meetings = 0;
    auto meet = [&](float mine, float& other) {
      const int at = (meetings & 1) * 2 * ROWS + row;
      s_meet[at + half * ROWS] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(met);
      if (!need(met, meetings)) return false;
      other = s_meet[at + (half ^ 1) * ROWS];
      ++meetings;
      return true;
    };
    int done = 0, seg = 0;  // done: parities only
    for (bool on = share > 0; on; on = go_on(cur, share, part)) {
      int tile;
      const int count = take(cur, share, tile);
      if (count == 0) continue;
      const int toks = tokens(cur);
      const bool in = t_in < toks, idle = !__any_sync(0xFFFFFFFFu, in);
      const int t_row = cur.rt * pp.per + t_in;
      const int all_see = cur.L + cur.rt * pp.per;
      const int sees = cur.L + t_row;  // the last row that this one sees
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < count; ++j) {
        const int n = done + j;
        const uint32_t t_s = tl + (NB == 2 ? (n & 1) * TK : 0);
        const uint32_t pfull = base + O_PFULL + 16 * (NQ == 2 ? q : n & 1);  // of the first step
        need(base + O_SFULL + 8 * (NQ == 2 ? q : n & 1), NQ == 2 ? n : n >> 1);
        if (!ok) continue;
        if (idle) {  // no row of the warp is the item's: whatever P is, nobody looks
          if (lane == 0 && APART) mbar_arrive(base + O_SFREE + 8 * q);
          // (the next S can be there before the other warps have handed over this P)
          if (APART && j > 0 && !need(base + O_ODONE + 8 * q, n - 1)) continue;
          if (lane == 0) {
            for (int sub = 0; sub < SUB; ++sub) mbar_arrive(pfull + 8 * sub);
          }
          continue;
        }
        tc_fence_after();
        const int j0 = (tile + j) * TK;
        uint32_t v[W / 32][32];  // the thread's scores of the row
#pragma unroll
        for (int c = 0; c < W / 32; ++c) tmem_ld32(t_s + half * W + c * 32, v[c]);
        tmem_wait_ld();
        if constexpr (APART) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(base + O_SFREE + 8 * q);
        }
        if (j0 + TK - 1 > all_see) {
          const int last = sees - j0 - half * W;
#pragma unroll
          for (int c = 0; c < W / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i > last) v[c][i] = 0xFF800000u;  // -inf
        }
        // P of 32 columns, in pairs, and their sum
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, m2 = make_float2(0.f, 0.f);
        auto powers = [&](int c, uint32_t (&w)[16]) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 e = fma2(make_float2(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), c2, m2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], e);
            w[i / 2] = pack16<BF16>(e.x, e.y);
          }
        };
        float mx;
        {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < W / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              x[(i >> 1) & 3] = fmaxf(x[(i >> 1) & 3], fmaxf(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])));
          mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        }
        if constexpr (H == 2) {
          // (P can lie where the other thread's S did: it has read that)
          tc_fence_before();
          float other;
          if (!meet(mx, other)) continue;
          tc_fence_after();
          mx = fmaxf(mx, other);
        }
        mx = mx * p.scale_log2 - ATTN_BASE_BELOW<BF16>;
        // P's place, and O, are free when the last product with V has ended: with P in the
        // place of S, this S was computed after it
        const bool grows = __any_sync(0xFFFFFFFFu, in && mx > m + 8.f);  // (rows past the item's hold anything)
        if ((APART || (NQ == 1 && grows)) && j > 0) {
          if (!need(base + O_ODONE + 8 * q, n - 1)) continue;
          tc_fence_after();
        }
        if (grows) {
          const float mn = fmaxf(m, mx);
          const float a = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= a;
          if (j > 0) {
#pragma unroll
            for (int c = half * (D / 16 / H); c < (half + 1) * (D / 16 / H); ++c) {
              uint32_t x[16];
              tmem_ld16(t_o + c * 16, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * a);
              tmem_st16(t_o + c * 16, x);
            }
          }
        }
        m2.x = m2.y = m == -INFINITY ? 0.f : -m;
        const uint32_t t_p = (APART ? tmem + ((uint32_t)((warp & 3) * 32) << 16) + COL_P + q * 64 : t_s) + half * (W / 2);
#pragma unroll
        for (int c = 0; c < W / 32; ++c) {
          uint32_t w[16];
          powers(c, w);
          tmem_st16(t_p + c * 16, w);
          if ((c + 1) % (W / 32 / SUB) == 0) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + 8 * (c / (W / 32 / SUB)));
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }

      // ------------------------------------------------ end of the segment
      if constexpr (H == 2) {
        float other = 0.f;
        if (ok && !idle) meet(l, other);
        l += other;
      }
      need(base + O_OLAST + 8 * q, seg);
      tc_fence_after();
      const bool last_tile = tile + count == cur.tiles, whole = tile == 0 && last_tile;
      if (tid == 0 && !last_tile)
        p.cuts[blockIdx.x] = make_int4(cur.first + cur.rt * pp.per, cur.h, toks * p.g, attn_cut(true, tile == 0));
      constexpr int PART = ROWS * (D + 2);
      float* partial = p.ws + ((int64_t)blockIdx.x * 2 + (tile == 0 ? 1 : 0)) * PART;
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
        constexpr int DH = D / H, STEP = DH < 64 ? DH : 64;  // columns of a thread
        uint32_t w[DH / 2];
#pragma unroll
        for (int c = 0; c < DH; c += STEP) {
          uint32_t v[STEP / 32][32];
#pragma unroll
          for (int i = 0; i < STEP / 32; ++i) tmem_ld32(t_o + half * DH + c + 32 * i, v[i]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < STEP; i += 2)
            w[(c + i) / 2] = pack16<BF16>(__uint_as_float(v[i >> 5][i & 31]) * inv, __uint_as_float(v[i >> 5][(i & 31) + 1]) * inv);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + O_OEMPTY + 8 * q);
        // Four lanes exchange their rows' 32 columns, so that they store a row's 64 bytes at a time.
        uint16_t* rows[4];
        bool have[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rows[k] = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)to16, (lane & 28) + k)) + half * DH + (lane & 3) * 8;
          have[k] = __shfl_sync(0xFFFFFFFFu, in && ok, (lane & 28) + k);
        }
#pragma unroll
        for (int c = 0; c < DH; c += 32) {
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
        if (ok && in && half == 0 && p.lse) p.lse[at * p.Hq + cur.h * p.g + i_row] = (m + log2f(l)) * 0.69314718055994531f;
        done += count;
        ++seg;
        continue;
      }
#pragma unroll 1
      for (int c = half * (D / H); c < (half + 1) * (D / H); c += 32) {
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
        float* to = partial + (row & ~7) * D + c + (lane & 7) * 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(to + k * D) = make_float4(a[k * 4], a[k * 4 + 1], a[k * 4 + 2], a[k * 4 + 3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + O_OEMPTY + 8 * q);
      if (whole) {
        if (ok && in && half == 0 && p.lse) p.lse[at * p.Hq + cur.h * p.g + i_row] = (m + log2f(l)) * 0.69314718055994531f;
      } else if (ok && half == 0) {
        partial[ROWS * D + row] = m;
        partial[ROWS * D + ROWS + row] = l;
      }
      done += count;
      ++seg;
    }
  }

  __syncthreads();
  if (tid == 0 && s_flag[0]) atomicOr(p.status, s_flag[0]);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(__shfl_sync(0xFFFFFFFFu, (uint32_t)s_flag[1], 0), 512);
  }
}

template <bool BF16, int D, int NQ>
cudaError_t prepare() {
  return cudaFuncSetAttribute(prompt_kernel<BF16, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, NQ>::BYTES);
}

template <bool BF16, int D, int NQ>
cudaError_t launch(const PromptParams& p, const void* kmap, const void* vmap, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.grid);
  cfg.blockDim = dim3(THREADS<NQ>);
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
