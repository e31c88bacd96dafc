// qmm_cache.cu -- the paged cache's handle and entry points (include/qmm.h), and
// the two kernels that move its rows: compaction of an accepted branch and
// copies of pages.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <new>
#include <unordered_set>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn.h"

using namespace qmm;

struct qmm_cache {
  qmm_cache_desc d;
  int device = 0;
  int sm_count = 0;
  int page_shift = 0;
  CUtensorMap kmap, vmap;   // the pools' rows
  float* ws = nullptr;      // partials of split attention items
  int4* cuts = nullptr;     // which items are split (behind ws)
  int* status = nullptr;    // device error word
  uint64_t wait_limit_ns = 2000000000ull;  // 2 s
};

namespace {

std::mutex g_mu;
std::unordered_set<qmm_cache*>& live_caches() {
  static std::unordered_set<qmm_cache*> s;
  return s;
}

bool is_live(qmm_cache* h) {
  if (!h) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  return live_caches().count(h) != 0;
}

void free_cache(qmm_cache* h) {
  int old = -1;
  cudaGetDevice(&old);
  if (old != h->device) cudaSetDevice(h->device);
  cudaFree(h->ws);
  cudaFree(h->status);
  if (old >= 0 && old != h->device) cudaSetDevice(old);
  delete h;
}

int check_current(const qmm_cache* h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device ? QMM_OK : QMM_ERR_DEVICE;
}

// ---------------------------------------------------------------- compaction
// One CTA column per sequence; its threads share the sequence's page offsets in
// shared memory, then each owns one 16-byte chunk of a head's row in one layer
// and pool and moves it for every accepted node in order.  A destination L + 1
// + j lies at or before its own source and every later source (path increases
// and path[j] >= j + 1), so a thread that reads up to BATCH sources before
// it writes their destinations never reads a row that it has overwritten.
// Bound by memory: a row is read and written once.  Measured: 64 sequences, 64
// layers, 20 heads of 128, up to 15 rows moved each: 100 us (6.3 TB/s, 92 % of a copy);
// one sequence, 16 layers: 2.7 us, a launch's latency.
constexpr int COMMIT_THREADS = 256;
constexpr int COMMIT_BATCH = 8;

struct CommitParams {
  uint16_t* k_pool;
  uint16_t* v_pool;
  int64_t layer_stride, page_stride, n_pages;
  const int32_t* table;
  int64_t ld_table;
  int table_width, page_shift;
  const int32_t* lens;
  const int32_t* path;
  int64_t ld_path;
  const int32_t* accept;
  int32_t* lens_out;
  int32_t* status;
  int T, Hkv, n_layers, chunks;  // chunks: 16-byte chunks of a row
};

__global__ void __launch_bounds__(COMMIT_THREADS) commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int64_t s_src[QMM_TREE_MAX_T], s_dst[QMM_TREE_MAX_T];
  __shared__ int s_n;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int L = p.lens[b];
  const int k = p.accept[2 * b];
  if (tid < 32) {
    // the moves of the sequence: page offsets of every row that changes place
    const int64_t cap = (int64_t)p.table_width << p.page_shift;
    bool ok = L >= 0 && k >= 0 && k < p.T && (int64_t)L + 1 + k <= cap;
    int n = 0;
    for (int j0 = 0; j0 < k && ok; j0 += 32) {
      const int j = j0 + tid;
      int64_t src = -1, dst = -1;
      bool good = true;
      if (j < k) {
        const int node = p.path[b * p.ld_path + j];
        const int prev = j > 0 ? p.path[b * p.ld_path + j - 1] : 0;
        good = node >= j + 1 && node > prev && node < p.T && (int64_t)L + node < cap;
        if (good && node != j + 1) {
          const int rs = L + node, rd = L + 1 + j, in = (1 << p.page_shift) - 1;
          const int ps = p.table[b * p.ld_table + (rs >> p.page_shift)];
          const int pd = p.table[b * p.ld_table + (rd >> p.page_shift)];
          good = ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages;
          src = ps * p.page_stride + (int64_t)(rs & in) * (p.chunks * 8);
          dst = pd * p.page_stride + (int64_t)(rd & in) * (p.chunks * 8);
        }
      }
      ok = __all_sync(0xFFFFFFFFu, good);
      const unsigned moves = __ballot_sync(0xFFFFFFFFu, good && src >= 0);
      if (src >= 0 && good) {
        const int at = n + __popc(moves & ((1u << tid) - 1));
        s_src[at] = src;
        s_dst[at] = dst;
      }
      n += __popc(moves);
    }
    if (tid == 0) {
      s_n = ok ? n : 0;
      if (blockIdx.x == 0) {
        p.lens_out[b] = ok ? L + 1 + k : L;
        if (!ok) atomicOr(p.status, DEV_ERR_INDEX);
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  const int64_t per = (int64_t)p.Hkv * p.chunks;
  const int64_t units = 2 * p.n_layers * per;
  const int64_t head = ((int64_t)p.chunks * 8) << p.page_shift;
  for (int64_t id = (int64_t)blockIdx.x * COMMIT_THREADS + tid; id < units && n > 0;
       id += (int64_t)gridDim.x * COMMIT_THREADS) {
    const int64_t lp = id / per;
    const int in = (int)(id - lp * per);
    uint16_t* base = (lp & 1 ? p.v_pool : p.k_pool) + (lp >> 1) * p.layer_stride + (in / p.chunks) * head +
                     (in % p.chunks) * 8;
    for (int j0 = 0; j0 < n; j0 += COMMIT_BATCH) {
      uint4 v[COMMIT_BATCH];
#pragma unroll
      for (int i = 0; i < COMMIT_BATCH; ++i)
        if (j0 + i < n) v[i] = *reinterpret_cast<const uint4*>(base + s_src[j0 + i]);
#pragma unroll
      for (int i = 0; i < COMMIT_BATCH; ++i)
        if (j0 + i < n) *reinterpret_cast<uint4*>(base + s_dst[j0 + i]) = v[i];
    }
  }
}

// ---------------------------------------------------------------- page copies
// Bound by memory: four 16-byte loads of a thread in flight.  Measured: 255 pages of
// 32 rows, 8 heads of 128, 64 layers: 464 us (6.9 TB/s, 102 % of a copy); 3 pages of
// 16 layers: 4.2 us.
constexpr int COPY_THREADS = 256;
constexpr int COPY_BATCH = 4;

struct CopyParams {
  uint16_t* k_pool;
  uint16_t* v_pool;
  int64_t layer_stride, page_stride, n_pages;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;
  int32_t* status;
  int Hkv, page_shift, chunks, pools;  // pools: of single layers, two each
};

// CTA (i, layer and pool; past 65,535 of these the next so many): the rows of a head are contiguous, rows * chunks
// 16-byte chunks; heads follow each other a page of rows apart.
__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ CopyParams p) {
  const int i = blockIdx.x;
  const int s = p.src[i], d = p.dst[i], page = 1 << p.page_shift;
  const int rows = p.rows ? p.rows[i] : page;
  if (s < 0 || s >= p.n_pages || d < 0 || d >= p.n_pages || rows < 0 || rows > page) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, DEV_ERR_INDEX);
    return;
  }
  if (s == d) return;
  const int per = rows * p.chunks, head = p.chunks << p.page_shift, total = p.Hkv * per;
  for (int lp = blockIdx.y; lp < p.pools; lp += gridDim.y) {
    uint16_t* base = (lp & 1 ? p.v_pool : p.k_pool) + (lp >> 1) * p.layer_stride;
    const uint4* from = reinterpret_cast<const uint4*>(base + s * p.page_stride);
    uint4* to = reinterpret_cast<uint4*>(base + d * p.page_stride);
    for (int at = threadIdx.x; at < total; at += COPY_THREADS * COPY_BATCH) {
      uint4 v[COPY_BATCH];
      int off[COPY_BATCH];
#pragma unroll
      for (int u = 0; u < COPY_BATCH; ++u) {
        const int x = at + u * COPY_THREADS;
        off[u] = x / per * head + x % per;
        if (x < total) v[u] = from[off[u]];
      }
#pragma unroll
      for (int u = 0; u < COPY_BATCH; ++u)
        if (at + u * COPY_THREADS < total) to[off[u]] = v[u];
    }
  }
}

// Whether the mma.sync kernel's warps work alone.  A warp alone ends a segment
// without the CTA's barriers and sums, but has one block of the cache in every
// unit where four warps share one.  So it is for many short sequences: more than
// three (sequence, head) pairs of 128 values (six of 64) for each CTA, and at most
// SOLO_MAX rows.  Measured, alone against shared, in us: 128 sequences of up to 30
// / 120 / 300 / 600 rows, 8 nodes, 20 heads of 128, two rows a node: 47 : 59, 61 :
// 91, 83 : 117, 120 : 145 (and since, with a shorter join, 120 rows: 51); 8 heads,
// one row: 16 : 23, 23 : 32, 31 : 41, 46 : 54.
// Past the limits: 48 sequences of up to 1,500 and 4,000 rows, 20 heads: 101 : 100,
// 223 : 216; 16 sequences of up to 120 and 600 rows: 23 : 17, 35 : 29.
// With 17 to 32 rows a head a warp walks the cache twice, and still ends before the
// tcgen05 kernel, whose segments are a longer chain, up to half as many rows: 128
// sequences of up to 30 / 120 / 300 rows, 20 heads of 128, 32 rows: 62 : 93, 87 :
// 122, 128 : 187; 24 rows, 8 heads: 29 : 42, 39 : 43, 54 : 80.  Past it: 800 rows,
// 265 : 223 and 107 : 96; with 64 rows a head and 10 heads, 30 / 120 / 300 rows: 73 :
// 55, 100 : 81, 131 : 124.
constexpr int SOLO_MAX = 1024;
bool attn_solo(const AttnParams& p, int64_t cap, int ctas, int D) {
  const int tiles = (p.R + attn_mma_tile_rows() - 1) / attn_mma_tile_rows();
  return tiles <= 2 && cap <= SOLO_MAX / tiles && (int64_t)p.B * p.Hkv * D >= (int64_t)3 * 128 * ctas;
}

}  // namespace

extern "C" {

int qmm_cache_create(qmm_cache_t* out, const qmm_cache_desc* d, void* stream) {
  if (!out) return QMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (!d || d->struct_size != sizeof(qmm_cache_desc) || !d->k_pool || !d->v_pool) return QMM_ERR_INVALID_ARG;
  if (d->dtype != QMM_DT_BF16 && d->dtype != QMM_DT_F16) return QMM_ERR_INVALID_ARG;
  if (d->n_layers < 1 || d->page_size < 16 || d->page_size > 1024 || (d->page_size & (d->page_size - 1)) ||
      d->n_kv_heads < 1 || d->n_kv_heads > 1024 || d->n_q_heads < d->n_kv_heads ||
      d->n_q_heads % d->n_kv_heads || d->n_q_heads / d->n_kv_heads > 64 ||
      (d->head_dim != 64 && d->head_dim != 128) || d->max_batch < 1 || d->max_batch > QMM_CACHE_MAX_BATCH ||
      d->n_pages < 1 || d->n_pages > INT32_MAX)
    return QMM_ERR_SHAPE;
  // tensor copies count the pools' rows in 32 bits
  const int64_t layer_rows = (int64_t)d->n_kv_heads * d->page_size;
  if (d->n_pages > INT32_MAX / layer_rows || d->n_layers > INT32_MAX / (d->n_pages * layer_rows)) return QMM_ERR_SHAPE;
  const int64_t pool_rows = d->n_layers * d->n_pages * layer_rows;
  if (((uintptr_t)d->k_pool | (uintptr_t)d->v_pool) & 15) return QMM_ERR_ALIGN;
  int dev = 0, sms = 0;
  const int rc = host_check_device(&dev, &sms);
  if (rc != QMM_OK) return rc;
  qmm_cache* h = new (std::nothrow) qmm_cache();
  if (!h) return host_cuda_fail(cudaErrorMemoryAllocation);
  h->d = *d;
  h->device = dev;
  h->sm_count = sms;
  while ((1 << h->page_shift) < d->page_size) ++h->page_shift;
  cudaStream_t st = (cudaStream_t)stream;
  // two partials of a CTA's largest row tile each
  const size_t rows_mma = (size_t)attn_mma_workers(sms, true) * attn_mma_tile_rows();
  const size_t rows_tc = (size_t)sms * attn_tc_tile_rows(INT32_MAX);
  const size_t part_bytes = 2 * (rows_mma > rows_tc ? rows_mma : rows_tc) * (d->head_dim + 2) * sizeof(float);
  const size_t ws_bytes = part_bytes + (size_t)attn_mma_workers(sms, true) * sizeof(int4);
  cudaError_t e = prepare_attn_mma(d->dtype == QMM_DT_BF16, d->head_dim);
  if (e == cudaSuccess) e = prepare_attn_tc(d->dtype == QMM_DT_BF16, d->head_dim);
  const bool f16 = d->dtype == QMM_DT_F16;
  if (e == cudaSuccess) e = host_pool_map(&h->kmap, d->k_pool, pool_rows, d->head_dim, 16, f16);
  if (e == cudaSuccess) e = host_pool_map(&h->vmap, d->v_pool, pool_rows, d->head_dim, 16, f16);
  void* ptr = nullptr;
  if (e == cudaSuccess && (e = host_dev_alloc(&ptr, ws_bytes)) == cudaSuccess)
    h->ws = static_cast<float*>(ptr), h->cuts = reinterpret_cast<int4*>(static_cast<char*>(ptr) + part_bytes);
  if (e == cudaSuccess && (e = host_dev_alloc(&ptr, sizeof(int))) == cudaSuccess)
    h->status = static_cast<int*>(ptr);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, sizeof(int), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    free_cache(h);
    return host_cuda_fail(e);
  }
  try {
    std::lock_guard<std::mutex> lk(g_mu);
    live_caches().insert(h);
  } catch (...) {
    free_cache(h);
    return host_cuda_fail(cudaErrorMemoryAllocation);
  }
  *out = h;
  return QMM_OK;
}

int qmm_cache_destroy(qmm_cache_t h) {
  if (!h) return QMM_OK;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!live_caches().erase(h)) return QMM_ERR_STATE;
  }
  free_cache(h);
  return QMM_OK;
}

int qmm_cache_sync_status(qmm_cache_t h, void* stream) {
  if (!is_live(h)) return QMM_ERR_STATE;
  cudaStream_t st = (cudaStream_t)stream;
  int word = 0;
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&word, h->status, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && word != 0) {
    e = cudaMemsetAsync(h->status, 0, sizeof(int), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) return host_cuda_fail(e);
  if (word & ~DEV_ERR_INDEX) return QMM_ERR_TIMEOUT;
  return word ? QMM_ERR_INDEX : QMM_OK;
}

int qmm_tree_attention(qmm_cache_t h, const qmm_attn_args* a, void* stream) {
  if (!is_live(h)) return QMM_ERR_STATE;
  if (!a || a->struct_size != sizeof(qmm_attn_args)) return QMM_ERR_INVALID_ARG;
  if (!a->q || !a->k_new || !a->v_new || !a->out || !a->page_table || !a->lens) return QMM_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !isfinite(a->scale)) return QMM_ERR_INVALID_ARG;
  const qmm_cache_desc& d = h->d;
  if (a->layer < 0 || a->layer >= d.n_layers || a->B < 1 || a->B > d.max_batch || a->T < 1 ||
      a->T > QMM_TREE_MAX_T || a->table_width < 1)
    return QMM_ERR_SHAPE;
  // rows are counted in 32 bits
  if (((int64_t)a->table_width << h->page_shift) > INT32_MAX - 4096) return QMM_ERR_SHAPE;
  if (((uintptr_t)a->q | (uintptr_t)a->k_new | (uintptr_t)a->v_new | (uintptr_t)a->out) & 15) return QMM_ERR_ALIGN;
  if ((((uintptr_t)a->lse | (uintptr_t)a->page_table | (uintptr_t)a->lens | (uintptr_t)a->n_tokens) & 3) ||
      ((uintptr_t)a->mask & 7))
    return QMM_ERR_ALIGN;
  // strides of dimensions with one entry are not followed
  const int dims[3][2] = {{a->B, a->B}, {a->T, a->T}, {d.n_q_heads, d.n_kv_heads}};
  for (int i = 0; i < 3; ++i)
    if ((dims[i][0] > 1 && ((a->q_stride[i] | a->out_stride[i]) & 7)) ||
        (dims[i][1] > 1 && ((a->k_stride[i] | a->v_stride[i]) & 7)))
      return QMM_ERR_ALIGN;
  if (a->B > 1 && (a->ld_table < a->table_width || (a->mask && a->ld_mask < a->T))) return QMM_ERR_ALIGN;
  int rc = check_current(h);
  if (rc != QMM_OK) return rc;

  AttnParams p;
  p.q = static_cast<const uint16_t*>(a->q);
  p.kn = static_cast<const uint16_t*>(a->k_new);
  p.vn = static_cast<const uint16_t*>(a->v_new);
  p.out = static_cast<uint16_t*>(a->out);
  p.q_sb = a->q_stride[0], p.q_st = a->q_stride[1], p.q_sh = a->q_stride[2];
  p.k_sb = a->k_stride[0], p.k_st = a->k_stride[1], p.k_sh = a->k_stride[2];
  p.v_sb = a->v_stride[0], p.v_st = a->v_stride[1], p.v_sh = a->v_stride[2];
  p.o_sb = a->out_stride[0], p.o_st = a->out_stride[1], p.o_sh = a->out_stride[2];
  p.lse = a->lse;
  p.page_stride = (int64_t)d.n_kv_heads * d.page_size * d.head_dim;
  p.n_pages = d.n_pages;
  p.k_pool = static_cast<uint16_t*>(d.k_pool) + a->layer * d.n_pages * p.page_stride;
  p.v_pool = static_cast<uint16_t*>(d.v_pool) + a->layer * d.n_pages * p.page_stride;
  p.table = a->page_table;
  p.ld_table = a->ld_table;
  p.table_width = a->table_width;
  p.page_shift = h->page_shift;
  p.lens = a->lens;
  p.n_tokens = a->n_tokens;
  p.mask = a->mask;
  p.ld_mask = a->ld_mask;
  p.B = a->B;
  p.T = a->T;
  p.Hq = d.n_q_heads;
  p.Hkv = d.n_kv_heads;
  p.g = d.n_q_heads / d.n_kv_heads;
  p.R = p.T * p.g;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.ws = h->ws;
  p.cuts = h->cuts;
  p.status = h->status;
  p.wait_limit_ns = h->wait_limit_ns;
  const bool bf16 = d.dtype == QMM_DT_BF16;
  const bool solo = attn_solo(p, (int64_t)a->table_width << h->page_shift, attn_mma_workers(h->sm_count, false),
                              d.head_dim);
  const bool tc = !solo && p.R > attn_mma_tile_rows();
  const int rows = tc ? attn_tc_tile_rows(p.R) : attn_mma_tile_rows();
  const int tk = tc ? attn_tc_tile_cache_rows() : attn_mma_tile_cache_rows(solo);
  p.RT = (p.R + rows - 1) / rows;
  p.grid = tc ? h->sm_count : attn_mma_workers(h->sm_count, solo);
  p.row0 = (int64_t)a->layer * d.n_pages * d.n_kv_heads * d.page_size;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = tc ? launch_attn_tc(p, bf16, d.head_dim, &h->kmap, &h->vmap, st)
                     : launch_attn_mma(p, bf16, d.head_dim, solo, st);
  // items of one unit each are never cut: nothing to join
  if (e == cudaSuccess && ((int64_t)a->table_width << h->page_shift) > tk)
    e = launch_attn_join(p, bf16, d.head_dim, tk, rows, h->sm_count, st);
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

int qmm_cache_commit(qmm_cache_t h, int B, int T, const int32_t* page_table, int64_t ld_table, int table_width,
                     const int32_t* lens, const int32_t* path, int64_t ld_path, const int32_t* accept,
                     int32_t* lens_out, void* stream) {
  if (!is_live(h)) return QMM_ERR_STATE;
  if (!page_table || !lens || !path || !accept || !lens_out || lens_out == lens) return QMM_ERR_INVALID_ARG;
  if (B < 1 || B > h->d.max_batch || T < 1 || T > QMM_TREE_MAX_T || table_width < 1) return QMM_ERR_SHAPE;
  if (((int64_t)table_width << h->page_shift) > INT32_MAX - 4096) return QMM_ERR_SHAPE;
  if (B > 1 && (ld_path < T || ld_table < table_width)) return QMM_ERR_ALIGN;
  if (((uintptr_t)page_table | (uintptr_t)lens | (uintptr_t)path | (uintptr_t)accept | (uintptr_t)lens_out) & 3)
    return QMM_ERR_ALIGN;
  const int rc = check_current(h);
  if (rc != QMM_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  CommitParams p;
  p.k_pool = static_cast<uint16_t*>(h->d.k_pool);
  p.v_pool = static_cast<uint16_t*>(h->d.v_pool);
  p.page_stride = (int64_t)h->d.n_kv_heads * h->d.page_size * h->d.head_dim;
  p.layer_stride = h->d.n_pages * p.page_stride;
  p.n_pages = h->d.n_pages;
  p.table = page_table;
  p.ld_table = ld_table;
  p.table_width = table_width;
  p.page_shift = h->page_shift;
  p.lens = lens;
  p.path = path;
  p.ld_path = ld_path;
  p.accept = accept;
  p.lens_out = lens_out;
  p.status = h->status;
  p.T = T;
  p.Hkv = h->d.n_kv_heads;
  p.n_layers = h->d.n_layers;
  p.chunks = h->d.head_dim / 8;
  const int64_t units = 2ll * p.n_layers * p.Hkv * p.chunks;
  int64_t x = (units + COMMIT_THREADS - 1) / COMMIT_THREADS;
  if (x > 65535) x = 65535;
  commit_kernel<<<dim3((unsigned)x, (unsigned)B), COMMIT_THREADS, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

int qmm_cache_copy(qmm_cache_t h, int n, const int32_t* src, const int32_t* dst, const int32_t* rows,
                   void* stream) {
  if (!is_live(h)) return QMM_ERR_STATE;
  if (n < 0 || n > (1 << 20)) return QMM_ERR_SHAPE;
  if (n == 0) return QMM_OK;
  if (!src || !dst) return QMM_ERR_INVALID_ARG;
  if (((uintptr_t)src | (uintptr_t)dst | (uintptr_t)rows) & 3) return QMM_ERR_ALIGN;
  const int rc = check_current(h);
  if (rc != QMM_OK) return rc;
  CopyParams p;
  p.k_pool = static_cast<uint16_t*>(h->d.k_pool);
  p.v_pool = static_cast<uint16_t*>(h->d.v_pool);
  p.page_stride = (int64_t)h->d.n_kv_heads * h->d.page_size * h->d.head_dim;
  p.layer_stride = h->d.n_pages * p.page_stride;
  p.n_pages = h->d.n_pages;
  p.src = src;
  p.dst = dst;
  p.rows = rows;
  p.status = h->status;
  p.Hkv = h->d.n_kv_heads;
  p.page_shift = h->page_shift;
  p.chunks = h->d.head_dim / 8;
  p.pools = 2 * h->d.n_layers;
  const unsigned y = p.pools < 65535 ? p.pools : 65535;
  copy_kernel<<<dim3((unsigned)n, y), COPY_THREADS, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMM_OK : host_cuda_fail(e);
}

int qmm_debug_set_cache_wait_limit(qmm_cache_t h, int64_t ns) {
  if (!is_live(h)) return QMM_ERR_STATE;
  if (ns < 0) return QMM_ERR_INVALID_ARG;
  h->wait_limit_ns = (uint64_t)ns;
  return QMM_OK;
}

}  // extern "C"
