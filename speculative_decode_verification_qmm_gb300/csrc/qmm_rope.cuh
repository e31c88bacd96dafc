// qmm_rope.cuh -- launch parameters of the kernel that turns heads by their
// positions (internal; qmm_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// Heads with a source and a destination of their own.  `pool`: rows lie in pages.
struct RopeHeads {
  const void* src;
  void* dst;
  int64_t s_seq, s_row, s_head;  // strides in elements; packed rows have no s_seq
  int64_t d_seq, d_row, d_head;
  int heads;
  int turned;
  int pool;
};

struct RopeParams {
  RopeHeads part[3];
  int parts;
  int heads;   // of all parts
  int D;       // of a head
  int m;       // turned pairs of a head
  int half;    // layout: pairs (i, i + m), else (2 i, 2 i + 1)
  float amplitude;
  const uint64_t* turns;
  // one position a row; NULL: lens[b] + i (packed rows)
  const int32_t* positions;
  int64_t rows;  // all rows of the call
  int T;         // rows of a sequence, where they are not packed
  // appended rows: packed, row i of sequence b is starts[b] + i
  int B;
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* table;
  int64_t ld_table;
  int table_width;
  int page_shift;
  int64_t page_stride, n_pages;
  int32_t* status;
};

// src_dt, dst_dt: QMM_DT_*; packed: rows are appended to a paged cache.
cudaError_t launch_rope(const RopeParams& p, int src_dt, int dst_dt, bool packed, int sms, cudaStream_t st);

}  // namespace qmm
