// qmm_rope.cu -- rotary positions (qmm_rotate) and, on the way into the paged
// cache, the same for appended rows (qmm_cache_append).
//
// Mathematics.  A pair (x, y) of a head's dimensions at position p becomes
//     A (x cos w - y sin w),  A (x sin w + y cos w),   w = 2 pi p f
// with f in turns a position.  Only p f modulo one turn matters, and p is whole:
// f is held as a 64-bit fraction of a turn, so that the wrapping integer product
// p * f is that remainder exactly, however far the position (in fp32 the angle of
// position 131,071 would be off by 0.008).  Its upper 32 bits, rounded, go to
// sincospi; what they lose is below 2^-25 turns.
//
// Work.  A unit is V dimensions of a head and the V that they are paired with.  A CTA takes
// up to 256 units of up to 32 rows: its threads work out the rows' sines and cosines once,
// for all heads, and each thread keeps its unit and walks the rows, a few of them in
// flight, the first ones requested before the angles are worked out.
// What bounds it: memory for many rows (8,192 rows of 40 + 20 + 20 heads of 128 from fp32 into
// a cache: 84 us, 6.0 TB/s, 89 % of a copy; 4,101 rows of 36 heads of 96, a quarter turned, 16
// bits: 12.9 us, 4.4 TB/s, of which a CTA's start takes a quarter), a launch for few (2.5 us).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"
#include "qmm_rope.cuh"

namespace qmm {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_ROWS = 32;      // of a CTA
constexpr int MAX_ANGLES = 2048;  // of a CTA
static_assert(MAX_ANGLES >= QMM_ROPE_MAX_DIM / 2, "a row's angles");

// V dimensions as they are in memory, and their values.
template <int DT, int V>
struct Raw {
  static constexpr int WORDS = DT == QMM_DT_F32 ? V : (V + 1) / 2;
  uint32_t w[WORDS];
};

template <int DT, int V>
__device__ __forceinline__ void load_vec(const char* at, Raw<DT, V>& r) {
  if constexpr (Raw<DT, V>::WORDS >= 4) {
#pragma unroll
    for (int i = 0; i < Raw<DT, V>::WORDS; i += 4) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(at) + i / 4);
      r.w[i] = v.x, r.w[i + 1] = v.y, r.w[i + 2] = v.z, r.w[i + 3] = v.w;
    }
  } else if constexpr (Raw<DT, V>::WORDS == 2) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(at));
    r.w[0] = v.x, r.w[1] = v.y;
  } else if constexpr (DT == QMM_DT_F32) {
    r.w[0] = __ldcs(reinterpret_cast<const uint32_t*>(at));
  } else {
    r.w[0] = __ldcs(reinterpret_cast<const uint16_t*>(at));
  }
}

template <int DT, int V>
__device__ __forceinline__ void values(const Raw<DT, V>& r, float (&x)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if constexpr (DT == QMM_DT_F32)
      x[e] = __uint_as_float(r.w[e]);
    else
      x[e] = unpack16<DT == QMM_DT_BF16>((uint16_t)(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2]));
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_vec(char* at, const float (&x)[V]) {
  if constexpr (DT == QMM_DT_F32) {
    float* p = reinterpret_cast<float*>(at);
    if constexpr (V == 1) {
      *p = x[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
  } else {
    constexpr bool BF = DT == QMM_DT_BF16;
    if constexpr (V == 1)
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)pack16<BF>(x[0], 0.f);
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(at) = make_uint2(pack16<BF>(x[0], x[1]), pack16<BF>(x[2], x[3]));
    else
      *reinterpret_cast<uint4*>(at) =
          make_uint4(pack16<BF>(x[0], x[1]), pack16<BF>(x[2], x[3]), pack16<BF>(x[4], x[5]), pack16<BF>(x[6], x[7]));
  }
}

// Units of a head, in order: the m / V turned ones (with V = 1 single pairs in either
// layout), then the rest, V dimensions each.  Interleaved with V > 1: V / 2 pairs in one
// vector, which has no second one.
template <int V>
__host__ __device__ __forceinline__ int units_of(const RopeParams& p) {
  return V > 1 && !p.half ? p.D / V : p.m / V + (p.D - 2 * p.m) / V;
}

template <int V>
__device__ __forceinline__ void unit_place(const RopeParams& p, int unit, int& first, int& second, int& pair, bool& turn) {
  if (V > 1 && !p.half) {
    first = unit * V, pair = first / 2, second = -1, turn = pair < p.m;
    return;
  }
  const int n = p.m / V;
  turn = unit < n;
  if (turn) {
    pair = unit * V;
    first = p.half ? pair : 2 * pair;
    second = p.half ? pair + p.m : 2 * pair + 1;
  } else {
    first = 2 * p.m + (unit - n) * V, second = -1, pair = 0;
  }
}

// A place that walks rows: `step` bytes from one to the next, `wrap` more behind the last row
// of a sequence.
struct Walk {
  int64_t step, wrap;
  int i, T;
  template <typename P>
  __device__ __forceinline__ void on(P*& at) {
    at += step;
    if (++i == T) i = 0, at += wrap;
  }
};

// grid: groups of `rows` rows, times groups of blockDim units.
template <int SRC, int DST, int V, bool PACKED>
__global__ void __launch_bounds__(THREADS, 3) rope_kernel(const __grid_constant__ RopeParams p, int rows) {
  constexpr int AHEAD = 4;  // rows in flight
  constexpr int SS = SRC == QMM_DT_F32 ? 4 : 2, DS = DST == QMM_DT_F32 ? 4 : 2;
  __shared__ float2 s_cs[MAX_ANGLES];
  __shared__ int64_t s_pool[MAX_ROWS];  // PACKED: the row's place in a pool, -1: none
  __shared__ int s_pos[MAX_ROWS];
  const int tid = threadIdx.x, threads = blockDim.x;
  const uint32_t row0 = blockIdx.x * (uint32_t)rows;
  const int n = p.rows - row0 < rows ? (int)(p.rows - row0) : rows;
  const uint32_t units = units_of<V>(p), total = p.heads * units;
  const uint32_t u = blockIdx.y * threads + tid;
  const bool mine = u < total;
  int h = mine ? u / units : 0, first = 0, second = -1, pair = 0, part = 0;
  bool turn = false;
  if (mine) {
    unit_place<V>(p, u - h * units, first, second, pair, turn);
    while (h >= p.part[part].heads) h -= p.part[part].heads, ++part;
  }
  const RopeHeads& t = p.part[part];
  turn = turn && t.turned;
  const bool two = second >= 0, pool = PACKED && t.pool;
  const int64_t other = two ? second - first : 0;
  const uint32_t b0 = PACKED ? 0 : row0 / (uint32_t)p.T, i0 = PACKED ? row0 : row0 - b0 * p.T;
  const char* src = static_cast<const char*>(t.src) + (b0 * t.s_seq + i0 * t.s_row + h * t.s_head + first) * SS;
  char* const dst0 = static_cast<char*>(t.dst) + (h * t.d_head + first) * DS;
  char* dst = dst0 + (b0 * t.d_seq + i0 * t.d_row) * DS;
  const int T = PACKED ? -1 : p.T;
  Walk from{t.s_row * SS, (t.s_seq - p.T * t.s_row) * SS, (int)i0, T};
  Walk to{t.d_row * DS, (t.d_seq - p.T * t.d_row) * DS, (int)i0, T};
  Raw<SRC, V> a[AHEAD], c[AHEAD];
  auto load = [&](int k) {
    load_vec<SRC, V>(src, a[k]);
    if (two) load_vec<SRC, V>(src + other * SS, c[k]);
    from.on(src);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (mine && k < n) load(k);
  if (tid < n) {
    const int64_t row = row0 + tid;
    if constexpr (PACKED) {
      // the sequence that the row is of; a row behind the last one is left alone
      int lo = 0, hi = p.B;
      while (lo < hi) {  // the number of sequences that end at or before the row
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.starts + mid + 1) <= row) lo = mid + 1;
        else hi = mid;
      }
      int64_t place = -1, at = 0;
      if (lo < p.B && row >= __ldg(p.starts + lo)) {
        const int L = __ldg(p.lens + lo);
        at = (int64_t)L + (row - __ldg(p.starts + lo));
        int page = -1;
        if (L >= 0 && at < ((int64_t)p.table_width << p.page_shift)) page = __ldg(p.table + lo * p.ld_table + (at >> p.page_shift));
        if (page >= 0 && page < p.n_pages)
          place = page * p.page_stride + (at & ((1 << p.page_shift) - 1)) * p.D;
        else if (blockIdx.y == 0)
          atomicOr(p.status, DEV_ERR_INDEX);
      }
      s_pool[tid] = place;
      s_pos[tid] = p.positions ? __ldg(p.positions + row) : (int)at;
    } else {
      s_pos[tid] = __ldg(p.positions + row);
    }
  }
  __syncthreads();
  for (uint32_t j = tid; j < (uint32_t)(n * p.m); j += threads) {
    const uint32_t r = j / (uint32_t)p.m;
    const uint64_t w = (uint64_t)(int64_t)s_pos[r] * __ldg(reinterpret_cast<const unsigned long long*>(p.turns) + (j - r * p.m));
    const int frac = (int)((w + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2 / 2^32: half turns
    s_cs[j] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
  if (!mine) return;
  const float2* cs = s_cs + pair;
  for (int r0 = 0; r0 < n; r0 += AHEAD) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int r = r0 + k;
      if (r >= n) break;
      float x[V], y[V];
      values<SRC, V>(a[k], x);
      if (two) values<SRC, V>(c[k], y);
      if (r + AHEAD < n) load(k);
      if (turn) {
        if (two) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 f = cs[e];
            const float v = x[e], w = y[e];
            x[e] = v * f.x - w * f.y;
            y[e] = v * f.y + w * f.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e + 1 < V; e += 2) {
            const float2 f = cs[e / 2];
            const float v = x[e], w = x[e + 1];
            x[e] = v * f.x - w * f.y;
            x[e + 1] = v * f.y + w * f.x;
          }
        }
      }
      cs += p.m;
      char* at = dst;
      to.on(dst);
      if constexpr (PACKED) {
        const int64_t place = s_pool[r];
        if (place < 0) continue;
        if (pool) at = dst0 + place * DS;
      }
      store_vec<DST, V>(at, x);
      if (two) store_vec<DST, V>(at + other * DS, y);
    }
  }
}

template <int SRC, int DST, int V, bool PACKED>
cudaError_t launch(const RopeParams& p, int sms, cudaStream_t st) {
  const int64_t total = (int64_t)p.heads * units_of<V>(p), groups = (total + THREADS - 1) / THREADS;
  const int threads = (int)((total + groups - 1) / groups + 31) / 32 * 32;
  // Rows of a CTA: many, since each CTA has its units to work out, but in whole waves.  (16 heads of
  // 128, bf16, us: 8,192 rows 13.7, always 32 rows 18.3, always 4 15.3; 1,000 rows 3.7, 12.6 and 4.0.)
  const int64_t most = p.m > 0 && MAX_ANGLES / p.m < MAX_ROWS ? MAX_ANGLES / p.m : MAX_ROWS;
  const int64_t slots = (int64_t)sms * (3 * THREADS / threads), all = p.rows * groups;
  const int64_t waves = (all + slots * most - 1) / (slots * most);
  int64_t rows = (all + slots * waves - 1) / (slots * waves);
  rows = rows > most ? most : rows;
  rope_kernel<SRC, DST, V, PACKED><<<dim3((unsigned)((p.rows + rows - 1) / rows), (unsigned)groups), threads, 0, st>>>(p, (int)rows);
  return cudaGetLastError();
}

template <int SRC, int DST, bool PACKED>
cudaError_t launch_v(const RopeParams& p, int sms, cudaStream_t st) {
  // Vectors of 16 bytes of the source, or four dimensions of 16 bits, where every one of them
  // lies on its boundary.  (fp32 with eight: 91 us for 8,192 rows of 40 + 20 + 20 heads, with
  // four 82; 16 bits, 8,192 rows of 16 heads: 13.7 with eight, 14.8 with four.)
  const int s = SRC == QMM_DT_F32 ? 4 : 2, d = DST == QMM_DT_F32 ? 4 : 2;
  int64_t bits = p.D | (p.half ? p.m : 2 * p.m);
  uintptr_t src = 0, dst = 0;
  for (int i = 0; i < p.parts; ++i) {
    const RopeHeads& t = p.part[i];
    bits |= t.s_seq | t.s_row | t.s_head | t.d_seq | t.d_row | t.d_head;
    src |= (uintptr_t)t.src, dst |= (uintptr_t)t.dst;
  }
  if constexpr (SRC != QMM_DT_F32)
    if (!(bits & 7) && !((src | dst) & 15)) return launch<SRC, DST, 8, PACKED>(p, sms, st);
  if (!(bits & 3) && !(src & (4 * s - 1)) && !(dst & (4 * d - 1))) return launch<SRC, DST, 4, PACKED>(p, sms, st);
  return launch<SRC, DST, 1, PACKED>(p, sms, st);
}

template <int SRC>
cudaError_t launch_src(const RopeParams& p, int dst_dt, bool packed, int sms, cudaStream_t st) {
  if (packed)
    return dst_dt == QMM_DT_BF16 ? launch_v<SRC, QMM_DT_BF16, true>(p, sms, st) : launch_v<SRC, QMM_DT_F16, true>(p, sms, st);
  switch (dst_dt) {
    case QMM_DT_BF16: return launch_v<SRC, QMM_DT_BF16, false>(p, sms, st);
    case QMM_DT_F16: return launch_v<SRC, QMM_DT_F16, false>(p, sms, st);
    default: return launch_v<SRC, QMM_DT_F32, false>(p, sms, st);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int src_dt, int dst_dt, bool packed, int sms, cudaStream_t st) {
  switch (src_dt) {
    case QMM_DT_BF16: return launch_src<QMM_DT_BF16>(p, dst_dt, packed, sms, st);
    case QMM_DT_F16: return launch_src<QMM_DT_F16>(p, dst_dt, packed, sms, st);
    default: return launch_src<QMM_DT_F32>(p, dst_dt, packed, sms, st);
  }
}

}  // namespace qmm

using namespace qmm;

int qmm::rope_check(const qmm_rope* r, int D) {
  if (!r || r->struct_size != sizeof(qmm_rope) || !r->turns) return QMM_ERR_INVALID_ARG;
  if (r->layout != QMM_ROPE_HALF && r->layout != QMM_ROPE_INTERLEAVED) return QMM_ERR_INVALID_ARG;
  if (!isfinite(r->amplitude)) return QMM_ERR_INVALID_ARG;
  if (r->dims < 2 || r->dims > D || (r->dims & 1)) return QMM_ERR_SHAPE;
  return (uintptr_t)r->turns & 7 ? QMM_ERR_ALIGN : QMM_OK;
}

extern "C" int qmm_rotate(const qmm_rotate_args* a, void* stream) {
  if (!a || a->struct_size != sizeof(qmm_rotate_args)) return QMM_ERR_INVALID_ARG;
  if (!a->x || !a->out || !a->positions || a->in_dtype > QMM_DT_F32 || a->out_dtype > QMM_DT_F32) return QMM_ERR_INVALID_ARG;
  if (a->head_dim < 2 || a->head_dim > QMM_ROPE_MAX_DIM || a->heads < 1 || a->heads > QMM_ROPE_MAX_HEADS || a->turned_heads < 0 ||
      a->turned_heads > a->heads || a->B < 1 || a->T < 1 || (int64_t)a->B * a->T > INT32_MAX)
    return QMM_ERR_SHAPE;
  int rc = rope_check(&a->rope, a->head_dim);
  if (rc != QMM_OK) return rc;
  const int se = a->in_dtype == QMM_DT_F32 ? 4 : 2, de = a->out_dtype == QMM_DT_F32 ? 4 : 2;
  if (((uintptr_t)a->x & (se - 1)) || ((uintptr_t)a->out & (de - 1)) || ((uintptr_t)a->positions & 3)) return QMM_ERR_ALIGN;
  // in place: every element is read by the thread that writes it, if it stays where it is
  const int n[3] = {a->B, a->T, a->heads};
  if (a->out == a->x) {
    if (se != de) return QMM_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && a->x_stride[i] != a->out_stride[i]) return QMM_ERR_INVALID_ARG;
  }
  int dev = 0, sms = 0;
  rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  RopeParams p = {};
  int64_t s[3], d[3];
  for (int i = 0; i < 3; ++i)  // strides of dimensions with one entry are not followed
    s[i] = n[i] > 1 ? a->x_stride[i] : 0, d[i] = n[i] > 1 ? a->out_stride[i] : 0;
  for (int k = 0; k < 2; ++k) {
    RopeHeads& t = p.part[k];
    const int first = k ? a->turned_heads : 0;
    t.src = static_cast<const char*>(a->x) + first * s[2] * se;
    t.dst = static_cast<char*>(a->out) + first * d[2] * de;
    t.s_seq = s[0], t.s_row = s[1], t.s_head = s[2];
    t.d_seq = d[0], t.d_row = d[1], t.d_head = d[2];
    t.heads = k ? a->heads - a->turned_heads : a->turned_heads;
    t.turned = !k;
  }
  p.parts = 2;
  p.heads = a->heads;
  p.D = a->head_dim;
  p.m = a->rope.dims / 2;
  p.half = a->rope.layout == QMM_ROPE_HALF;
  p.amplitude = a->rope.amplitude;
  p.turns = a->rope.turns;
  p.positions = a->positions;
  p.rows = (int64_t)a->B * a->T;
  p.T = a->T;
  const cudaError_t e = launch_rope(p, a->in_dtype, a->out_dtype, false, sms, (cudaStream_t)stream);
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}
