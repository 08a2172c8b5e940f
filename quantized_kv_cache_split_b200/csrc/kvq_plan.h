// Internal interface of the page planner (kvq_plan.cu).
#pragma once

#include "kvq_internal.h"

namespace kvq {

struct PlanArgs {
  int batch, page_size, num_pages, max_pages, max_tokens;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* page_table;
  int32_t* seq_lens_out;
  int32_t* free_count_out;
  int32_t* token_offsets;
  int32_t* slots;
  int32_t* positions;  // or null
  uint32_t* flags;
};

int launch_plan(const PlanArgs& a, cudaStream_t stream);

}  // namespace kvq
