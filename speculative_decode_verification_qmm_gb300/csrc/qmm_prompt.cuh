// qmm_prompt.cuh -- launch parameters of the prompt attention (internal; qmm_prompt.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm_attn.cuh"

namespace qmm {

// Rows are packed: q_st, o_st are strides of a row; T, R, RT, mask, n_tokens and the
// new rows' pointers have no part.  cuts: first row of the item, head, its rows, attn_cut.
struct PromptParams {
  AttnParams a;
  const int32_t* starts;
  int N;     // rows of q and out
  int rows;  // rows of a row tile: 128 or 256
  int per;   // tokens of a row tile: rows / g
};

int prompt_tile_cache_rows();
cudaError_t prepare_prompt(bool bf16, int D);
cudaError_t launch_prompt(const PromptParams& p, bool bf16, int D, const void* kmap, const void* vmap, cudaStream_t st);

}  // namespace qmm
