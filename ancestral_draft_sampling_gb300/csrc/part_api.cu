// part_api.cu -- the C ABI of what reads part of the cache (include/dspark.h):
// bounds of pages and their selection.
#include <cmath>

#include "cache_check.cuh"
#include "select_pages.cuh"

namespace {

using namespace dspark;

size_t align_up(size_t x, size_t n) { return (x + n - 1) / n * n; }

// The workspace of the selection: the scores of every list, the exact ones of
// many pages near the border, and what bounds the scores' errors.
struct SelectLayout {
  int stride, chunks;
  size_t border, reach_q, reach_k, total;
};

SelectLayout select_layout(const dspark_cache& c, int B, int lists) {
  SelectLayout L;
  L.stride = (c.max_pages + 3) / 4 * 4;
  L.chunks = (c.max_pages + kScoreChunk - 1) / kScoreChunk;
  const size_t rows = (size_t)B * lists * c.kv_heads;
  L.border = align_up(rows * L.stride * sizeof(float), 256);
  L.reach_q = align_up(L.border + rows * L.stride * sizeof(double), 256);
  L.reach_k = align_up(L.reach_q + rows * sizeof(float), 256);
  L.total = align_up(L.reach_k + (size_t)B * c.kv_heads * L.chunks * sizeof(float), 256);
  return L;
}

dspark_status select_sizes(const dspark_cache* c, int B, int T) {
  if (B <= 0 || T <= 0) return DSPARK_ERR_INVALID_ARG;
  if (B > DSPARK_CACHE_MAX_B || T > DSPARK_TREE_MAX_TOKENS ||
      (long long)B * c->kv_heads * ((c->max_pages + kScoreChunk - 1) / kScoreChunk) >= (1LL << 31))
    return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

}  // namespace

extern "C" {

dspark_status dspark_cache_bounds(const dspark_cache* cache, const int32_t* seq,
                                  const int32_t* start, const int32_t* length, int B, void* bounds,
                                  cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st != DSPARK_OK) return st;
  if (!start || !length || !bounds || !is4(seq) || !is4(start) || !is4(length) ||
      !aligned_to(bounds, 16))
    return DSPARK_ERR_INVALID_ARG;
  BoundsArgs a{};
  a.c = *cache;
  a.seq = seq;
  a.start = start;
  a.length = length;
  a.B = B;
  a.bounds = static_cast<char*>(bounds);
  return from_cuda(launch_cache_bounds(a, sm_count(), stream));
}

size_t dspark_select_workspace_bytes(const dspark_cache* cache, int B, int T, int shared) {
  if (check_cache(cache) != DSPARK_OK || select_sizes(cache, B, T) != DSPARK_OK) return 0;
  return select_layout(*cache, B, shared ? 1 : T).total;
}

dspark_status dspark_select_pages(const dspark_cache* cache, int layer, const int32_t* seq,
                                  const int32_t* length, const int32_t* token_count, const void* q,
                                  const void* bounds, int count, int first, int last, int shared,
                                  int B, int T, int heads, int32_t* pages, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st == DSPARK_OK) st = check_heads(heads, cache->kv_heads);
  if (st != DSPARK_OK) return st;
  if (!length || !q || !bounds || !pages || T <= 0 || layer < 0 || layer >= cache->layers ||
      count <= 0 || first < 0 || last < 0 || first > count || last > count - first)
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(bounds, 16)) return DSPARK_ERR_INVALID_ARG;
  const void* p4[] = {seq, length, token_count, pages};
  for (const void* p : p4)
    if (!is4(p)) return DSPARK_ERR_INVALID_ARG;
  st = select_sizes(cache, B, T);
  if (st == DSPARK_OK && heads / cache->kv_heads > DSPARK_TREE_MAX_GROUP) st = DSPARK_ERR_UNSUPPORTED;
  if (st != DSPARK_OK) return st;
  const int lists = shared ? 1 : T;
  const SelectLayout L = select_layout(*cache, B, lists);
  if (!workspace || workspace_bytes < L.total || !aligned_to(workspace, 256))
    return DSPARK_ERR_WORKSPACE;
  SelectArgs a{};
  a.c = *cache;
  a.layer = layer;
  a.seq = seq;
  a.length = length;
  a.tokens = token_count;
  a.q = static_cast<const char*>(q);
  a.bounds = static_cast<const char*>(bounds);
  a.count = count;
  a.first = first;
  a.last = last;
  a.lists = lists;
  a.B = B;
  a.T = T;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.pages = pages;
  a.stride = L.stride;
  a.chunks = L.chunks;
  char* ws = static_cast<char*>(workspace);
  a.scores = reinterpret_cast<float*>(ws);
  a.border = reinterpret_cast<double*>(ws + L.border);
  a.reach_q = reinterpret_cast<float*>(ws + L.reach_q);
  a.reach_k = reinterpret_cast<float*>(ws + L.reach_k);
  return from_cuda(launch_select_pages(a, sm_count(), stream));
}

}  // extern "C"
