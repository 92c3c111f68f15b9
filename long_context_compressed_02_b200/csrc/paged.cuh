// Between the translation units of the paged attention.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include "batch.cuh"
#include "../../include/csa.h"

namespace csa {

// A paged call as the pair kernel takes it (D = 512, bf16 rows).
struct PairParams {
  const void* q;                // [n_tok, H, 512]
  const int32_t* cu_q;
  const int64_t* q_pos;
  int n_seq, H;
  int64_t n_tok;
  const void* rows[2];          // page stores: 0 raw rows, 1 entries (null: none)
  PageTable pt[2];
  int64_t cap[2];               // rows that the tables can name
  int W, m;
  const float* sink;
  float scale_log2;
  void* out;
  int out_bf16;
};

// Whether launch_paged_pair takes pages of this size.
inline bool pair_page_size(int page_size) { return page_size >= 16; }
csa_status_t launch_paged_pair(PairParams& p, cudaStream_t st);

}  // namespace csa
