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
// Work.  A CTA takes the heads of one row, or a share of them where there are few
// rows: its threads work out the row's sines and cosines once, for all heads,
// and then each turns vectors of V dimensions.  Loads are issued before the angles
// are worked out.
// What bounds it: memory.
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
constexpr int MAX_PAIRS = QMM_ROPE_MAX_DIM / 2;
constexpr int AHEAD = 4;  // units of a thread whose loads are in flight

template <int DT>
struct Elem {
  using type = uint16_t;
};
template <>
struct Elem<QMM_DT_F32> {
  using type = float;
};

template <int DT, int V>
__device__ __forceinline__ void load_vec(const void* base, int64_t at, float (&x)[V]) {
  if constexpr (DT == QMM_DT_F32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (V == 4) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      x[0] = __ldcs(p);
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (V == 4) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
      x[0] = unpack16<DT == QMM_DT_BF16>((uint16_t)v.x), x[1] = unpack16<DT == QMM_DT_BF16>((uint16_t)(v.x >> 16));
      x[2] = unpack16<DT == QMM_DT_BF16>((uint16_t)v.y), x[3] = unpack16<DT == QMM_DT_BF16>((uint16_t)(v.y >> 16));
    } else {
      x[0] = unpack16<DT == QMM_DT_BF16>(*p);
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&x)[V]) {
  if constexpr (DT == QMM_DT_F32) {
    float* p = static_cast<float*>(base) + at;
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *p = x[0];
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p) =
          make_uint2(pack16<DT == QMM_DT_BF16>(x[0], x[1]), pack16<DT == QMM_DT_BF16>(x[2], x[3]));
    else
      *p = (uint16_t)pack16<DT == QMM_DT_BF16>(x[0], 0.f);
  }
}

// A unit of a head: V dimensions and, where they are turned, the V that they are
// paired with.  Units of a head, in order: the m / V turned ones (with V = 1 single
// pairs in either layout), then the rest, V dimensions each.  Interleaved with V = 4:
// two pairs in one vector, which has no second one.
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

template <int SRC, int DST, int V, bool PACKED>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 s_cs[MAX_PAIRS];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  int b = 0, i = 0;          // sequence, row in it
  int64_t pool_at = 0;       // of the row, in a pool
  int pos;
  if constexpr (PACKED) {
    // the sequence that the row is of; a row behind the last one is left alone
    int lo = 0, hi = p.B;
    while (lo < hi) {  // the number of sequences that end at or before the row
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.starts + mid + 1) <= row) lo = mid + 1;
      else hi = mid;
    }
    if (lo >= p.B || row < __ldg(p.starts + lo)) return;
    b = lo;
    i = (int)(row - __ldg(p.starts + b));
    const int L = __ldg(p.lens + b);
    const int64_t at = (int64_t)L + i;
    if (L < 0 || at >= ((int64_t)p.table_width << p.page_shift)) {
      if (tid == 0) atomicOr(p.status, DEV_ERR_INDEX);
      return;
    }
    const int page = __ldg(p.table + b * p.ld_table + (at >> p.page_shift));
    if (page < 0 || page >= p.n_pages) {
      if (tid == 0) atomicOr(p.status, DEV_ERR_INDEX);
      return;
    }
    pool_at = page * p.page_stride + (at & ((1 << p.page_shift) - 1)) * p.D;
    pos = p.positions ? __ldg(p.positions + row) : (int)at;
  } else {
    b = (int)(row / p.T);
    i = (int)(row - (int64_t)b * p.T);
    pos = __ldg(p.positions + row);
  }
  const int units = V > 1 && !p.half ? p.D / V : p.m / V + (p.D - 2 * p.m) / V;
  // a unit of a head that is not turned is the same places, copied
  const int total = p.heads * units, step = gridDim.y * THREADS;
  bool ready = p.m == 0;
  for (int u0 = blockIdx.y * THREADS + tid; __syncthreads_or(u0 < total); u0 += step * AHEAD) {
    float x[AHEAD][V], y[AHEAD][V];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int u = u0 + k * step;
      if (u >= total) continue;
      int h = u / units, first, second, pair;
      bool turn;
      unit_place<V>(p, u - h * units, first, second, pair, turn);
      int part = 0;
      while (h >= p.part[part].heads) h -= p.part[part].heads, ++part;
      const RopeHeads& t = p.part[part];
      const int64_t at = (PACKED ? row * t.s_row : b * t.s_seq + i * t.s_row) + h * t.s_head;
      load_vec<SRC, V>(t.src, at + first, x[k]);
      if (second >= 0) load_vec<SRC, V>(t.src, at + second, y[k]);
    }
    if (!ready) {
      for (int j = tid; j < p.m; j += THREADS) {
        const uint64_t w = (uint64_t)(int64_t)pos * __ldg(reinterpret_cast<const unsigned long long*>(p.turns) + j);
        const int frac = (int)((w + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2 / 2^32: half turns
        s_cs[j] = make_float2(c * p.amplitude, s * p.amplitude);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int u = u0 + k * step;
      if (u >= total) continue;
      int h = u / units, first, second, pair;
      bool turn;
      unit_place<V>(p, u - h * units, first, second, pair, turn);
      int part = 0;
      while (h >= p.part[part].heads) h -= p.part[part].heads, ++part;
      const RopeHeads& t = p.part[part];
      if (turn && t.turned) {
        if (second >= 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 cs = s_cs[pair + e];
            const float a = x[k][e], c = y[k][e];
            x[k][e] = a * cs.x - c * cs.y;
            y[k][e] = a * cs.y + c * cs.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e + 1 < V; e += 2) {
            const float2 cs = s_cs[pair + e / 2];
            const float a = x[k][e], c = x[k][e + 1];
            x[k][e] = a * cs.x - c * cs.y;
            x[k][e + 1] = a * cs.y + c * cs.x;
          }
        }
      }
      const int64_t at = (PACKED ? (t.pool ? pool_at : row * t.d_row) : b * t.d_seq + i * t.d_row) + h * t.d_head;
      store_vec<DST, V>(t.dst, at + first, x[k]);
      if (second >= 0) store_vec<DST, V>(t.dst, at + second, y[k]);
    }
  }
}

template <int SRC, int DST, int V, bool PACKED>
cudaError_t launch(const RopeParams& p, int sms, cudaStream_t st) {
  const int units = V > 1 && !p.half ? p.D / V : p.m / V + (p.D - 2 * p.m) / V;
  const int64_t total = (int64_t)p.heads * units;
  // shares of a row: one unit a thread where the rows alone do not fill the GPU
  int64_t most = (total + THREADS - 1) / THREADS, y = (4ll * sms + p.rows - 1) / p.rows;
  if (y > most) y = most;
  if (y > 65535) y = 65535;
  if (y < 1) y = 1;
  rope_kernel<SRC, DST, V, PACKED><<<dim3((unsigned)p.rows, (unsigned)y), THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <int SRC, int DST, bool PACKED>
cudaError_t launch_v(const RopeParams& p, int sms, cudaStream_t st) {
  // Vectors of four where every one of them lies on its boundary.
  const int s = SRC == QMM_DT_F32 ? 4 : 2, d = DST == QMM_DT_F32 ? 4 : 2;
  int64_t bits = p.D | (p.half ? p.m : 2 * p.m);
  bool wide = true;
  for (int i = 0; i < p.parts; ++i) {
    const RopeHeads& t = p.part[i];
    bits |= t.s_seq | t.s_row | t.s_head | t.d_seq | t.d_row | t.d_head;
    wide = wide && !((uintptr_t)t.src & (4 * s - 1)) && !((uintptr_t)t.dst & (4 * d - 1));
  }
  return wide && !(bits & 3) ? launch<SRC, DST, 4, PACKED>(p, sms, st) : launch<SRC, DST, 1, PACKED>(p, sms, st);
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
