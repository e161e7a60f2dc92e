// select_pages.cuh -- the arguments of the selection of pages.
#pragma once

#include "cache.cuh"

namespace dspark {

constexpr int kReachPages = 8;  // pages that SelectArgs::reach_k goes by

struct SelectArgs {
  dspark_cache c;
  int layer;
  const int32_t *seq, *length, *tokens;
  const char *q, *bounds;
  int count, first, last;
  int lists;   // of a sequence and key head: T, or 1 for all tokens together
  int B, T, heads, group;
  int32_t* pages;
  // workspace: [B][lists][kv_heads] rows
  int stride;      // pages of a row
  float* scores;   // [rows][stride]
  uint64_t* border;  // [rows][stride], the exact scores of many pages near the border
  float* reach_q;  // [B][T][kv_heads] the largest sum of |q| of a token's heads
  float* reach_k;  // [B][kv_heads][reaches] the largest |bound| of kReachPages pages
  int reaches;
  float error;     // of a score, relative to those two
};

cudaError_t launch_select_pages(const SelectArgs& a, int sms, cudaStream_t stream);

}  // namespace dspark
