// qmm_attn.h -- host launchers of the paged-cache and sampling kernels (internal),
// and the host helpers that qmm_api.cu lends them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

struct AttnParams;

// qmm_api.cu: allocation with the fault-injection hook, the device check, and
// the record behind qmm_last_cuda_error(NULL).
cudaError_t host_dev_alloc(void** p, size_t bytes);
int host_check_device(int* dev, int* sms);
int host_cuda_fail(cudaError_t e);

// A tensor map over the rows of a pool ([rows][D] 16-bit values): boxes of 64
// columns x box_rows rows, 128-byte swizzle.  map: a CUtensorMap.
cudaError_t host_pool_map(void* map, const void* base, int64_t rows, int D, int box_rows, bool f16);

// Rows of an item's tile for R rows, and cache rows of a unit.  mma.sync kernel:
// two CTAs per SM; solo: each warp works alone, for many short items.
constexpr int ATTN_MMA_CTAS_PER_SM = 2;
int attn_mma_tile_rows();
int attn_mma_tile_cache_rows(bool solo);
int attn_mma_workers(int sms, bool solo);  // AttnParams::grid
cudaError_t prepare_attn_mma(bool bf16, int D);
cudaError_t launch_attn_mma(const AttnParams& p, bool bf16, int D, bool solo, cudaStream_t st);

// tcgen05 kernel (more rows than the mma.sync kernel's tile), one CTA per SM; kmap, vmap: host_pool_map with boxes of 16 rows.
int attn_tc_tile_rows(int R);
int attn_tc_tile_cache_rows();
cudaError_t prepare_attn_tc(bool bf16, int D);
cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int D, const void* kmap, const void* vmap,
                           cudaStream_t st);

// Sums of the partials that a launch with those tiles left (qmm_attn_join.cu).
cudaError_t launch_attn_join(const AttnParams& p, bool bf16, int D, int tk, int rows, int sms, cudaStream_t st);

// The same for the prompt attention, by at most ATTN_PROMPT_GRID_MAX CTAs: rows a row tile.
constexpr int ATTN_PROMPT_GRID_MAX = 160;
cudaError_t launch_prompt_join(const AttnParams& p, bool bf16, int D, int rows, int sms, cudaStream_t st);

// Whether a description of rotary positions fits heads of D (qmm_rope.cu).
int rope_check(const qmm_rope* r, int D);

}  // namespace qmm
