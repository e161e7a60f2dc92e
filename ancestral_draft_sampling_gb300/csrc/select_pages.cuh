// select_pages.cuh -- the arguments of the selection of pages.
#pragma once

#include "cache.cuh"

namespace dspark {

constexpr int kScoreChunk = 64;  // pages that a warp scores for a key head

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
  double* border;  // [rows][stride], the exact scores of many pages near the border
  float* reach_q;  // [rows] the largest sum of |q|
  float* reach_k;  // [B][kv_heads][chunks] the largest |bound| of a chunk
  int chunks;
};

cudaError_t launch_select_pages(const SelectArgs& a, int sms, cudaStream_t stream);

}  // namespace dspark
