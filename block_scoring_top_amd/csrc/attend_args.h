// Arguments of the attention kernels (plain C++: shared by the host layer).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace idxk {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *kv_indptr, *kv_indices;
  const int32_t* kv_len;
  const int32_t* row_req;     // single tokens: or NULL
  const int32_t* tok_indptr;  // prompt tokens
  const int32_t* ids;         // single tokens: or NULL
  const float* slopes;        // or NULL
  uint16_t* out;
  float *part_o, *part_ml;    // rows split over workgroups: sums, (max, sum of weights)
  int64_t n_indices;
  int R, B, Hq, Hkv, n_pages, max_pages, page_size, K;
  float score_scale;          // times log2(e) unless the scores are capped
  float softcap;              // 0: none
};

// Tiles of 64 tokens per workgroup, and workgroups per row; rows of a workgroup where
// packed tokens share one.
struct AttnSplit {
  int chunk, splits, rows;
};

}  // namespace idxk
