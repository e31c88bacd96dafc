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

// mma.sync kernel: rows of an item's tile for R rows, and two CTAs per SM.
constexpr int ATTN_MMA_CTAS_PER_SM = 2;
int attn_mma_tile_rows(int R);
cudaError_t prepare_attn_mma(bool bf16, int D);
cudaError_t launch_attn_mma(const AttnParams& p, bool bf16, int D, int ctas, cudaStream_t st);


// tcgen05 kernel (more rows than the mma.sync kernel's tile holds), one CTA per SM.
int attn_tc_tile_rows(int R);
cudaError_t prepare_attn_tc(bool bf16, int D);
cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int D, int ctas, cudaStream_t st);

}  // namespace qmm
