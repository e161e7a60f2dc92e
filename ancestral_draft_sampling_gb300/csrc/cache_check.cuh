// cache_check.cuh -- the argument checks that the entry points of the cache
// share.
#pragma once

#include "cache.cuh"
#include "host_util.cuh"

namespace dspark {

inline bool is4(const void* p) { return aligned_to(p, 4); }

// The checks that every call on a cache makes.
inline dspark_status check_cache(const dspark_cache* c) {
  if (!c || !c->pool || !c->block_table || !c->page_count || !c->ref_count ||
      !c->free_list || !c->control)
    return DSPARK_ERR_INVALID_ARG;
  if (c->dtype != DSPARK_F32 && c->dtype != DSPARK_BF16) return DSPARK_ERR_INVALID_ARG;
  if (c->layers <= 0 || c->num_pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0 ||
      c->head_dim <= 0 || c->max_seqs <= 0 || c->max_pages <= 0)
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned_to(c->pool, 16) || !aligned_to(c->control, 16) || !is4(c->block_table) ||
      !is4(c->page_count) || !is4(c->ref_count) || !is4(c->free_list))
    return DSPARK_ERR_INVALID_ARG;
  if (c->layers > 1024 || c->page_size > 4096 || c->kv_heads > 1024 ||
      c->head_dim > 256 || c->head_dim % 8 != 0 ||
      (long long)c->max_seqs * c->max_pages >= (1LL << 31) ||
      (long long)c->max_pages * c->page_size > (1LL << 30))
    return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

inline dspark_status check_batch(int B) {
  if (B <= 0) return DSPARK_ERR_INVALID_ARG;
  return B > DSPARK_CACHE_MAX_B ? DSPARK_ERR_UNSUPPORTED : DSPARK_OK;
}

inline dspark_status check_heads(int heads, int kv_heads) {
  if (heads <= 0 || heads % kv_heads != 0) return DSPARK_ERR_INVALID_ARG;
  return DSPARK_OK;
}

}  // namespace dspark
