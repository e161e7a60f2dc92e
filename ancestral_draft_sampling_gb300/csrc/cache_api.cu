// cache_api.cu -- the C ABI of the paged key/value cache and the attention
// over it (include/dspark.h): argument checks and launches.
#include <cmath>

#include "cache.cuh"
#include "dspark_common.cuh"
#include "host_util.cuh"
#include "tree_attention.cuh"

namespace {

using namespace dspark;

bool is4(const void* p) { return aligned_to(p, 4); }

// The checks that every call on a cache makes.
dspark_status check_cache(const dspark_cache* c) {
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

dspark_status check_batch(int B) {
  if (B <= 0) return DSPARK_ERR_INVALID_ARG;
  return B > DSPARK_CACHE_MAX_B ? DSPARK_ERR_UNSUPPORTED : DSPARK_OK;
}

dspark_status check_heads(int heads, int kv_heads) {
  if (heads <= 0 || heads % kv_heads != 0) return DSPARK_ERR_INVALID_ARG;
  return DSPARK_OK;
}

// Whether one of n rows of `row` bytes, `step` (>= row) bytes apart, has a byte
// of the `bytes` ones at `to`.  The rows of a token are parts of a projection's
// output, and what lies between them is not theirs.
bool rows_meet(const void* rows, __int128 step, __int128 row, __int128 n, const void* to,
               __int128 bytes) {
  const __int128 from = reinterpret_cast<uintptr_t>(rows), at = reinterpret_cast<uintptr_t>(to);
  // the first row that ends behind `at`
  const __int128 i = from + row > at ? 0 : (at - from - row) / step + 1;
  return i < n && from + i * step < at + bytes;
}

// The workspace of the attention: what the merge has to do, then the partial
// results, two a block; no kernel has larger units than the tensor-core one.
struct TreeLayout {
  size_t part, total;
};

TreeLayout tree_layout(int T, int group, int D) {
  TreeLayout L;
  L.part = align_up((size_t)2 * kTreeMaxBlocks * sizeof(TreeJoin), 256);
  const int fit = 2 * (kTreeRows / group);  // drafted tokens of a tensor-core unit
  size_t rows = (size_t)(T < fit ? T : fit) * group * 2 * kTreeMaxBlocks;
  L.total = align_up(L.part + rows * (D + 2) * sizeof(float), 256);
  return L;
}

bool tree_sizes(int B, int T, int heads, int kv_heads, int D) {
  return B >= 1 && B <= DSPARK_CACHE_MAX_B && T >= 1 && T <= DSPARK_TREE_MAX_TOKENS &&
         kv_heads >= 1 && kv_heads <= 1024 && heads >= 1 && heads % kv_heads == 0 &&
         heads / kv_heads <= DSPARK_TREE_MAX_GROUP && D >= 8 && D <= 256 && D % 8 == 0;
}

}  // namespace

extern "C" {

dspark_status dspark_cache_init(const dspark_cache* cache, cudaStream_t stream) {
  const dspark_status st = check_cache(cache);
  return st != DSPARK_OK ? st : from_cuda(launch_cache_init(*cache, stream));
}

dspark_status dspark_cache_reserve(const dspark_cache* cache, const int32_t* seq,
                                   const int32_t* length, int tokens, int B,
                                   cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st != DSPARK_OK) return st;
  if (!length || !is4(length) || !is4(seq) || tokens < 0) return DSPARK_ERR_INVALID_ARG;
  return from_cuda(launch_cache_reserve(*cache, seq, length, tokens, B, stream));
}

dspark_status dspark_cache_release(const dspark_cache* cache, const int32_t* seq, int B,
                                   cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st != DSPARK_OK) return st;
  if (!is4(seq)) return DSPARK_ERR_INVALID_ARG;
  return from_cuda(launch_cache_release(*cache, seq, B, stream));
}

dspark_status dspark_cache_fork(const dspark_cache* cache, const int32_t* parent,
                                const int32_t* child, const int32_t* length, int B,
                                cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st != DSPARK_OK) return st;
  if (!parent || !child || !length || !is4(parent) || !is4(child) || !is4(length))
    return DSPARK_ERR_INVALID_ARG;
  return from_cuda(launch_cache_fork(*cache, parent, child, length, B, stream));
}

dspark_status dspark_cache_accept(const dspark_cache* cache, const int32_t* seq,
                                  const int32_t* length, const int32_t* accepted_len,
                                  const int32_t* path, int path_width, int extra,
                                  int tokens, int B, int32_t* new_length,
                                  cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st != DSPARK_OK) return st;
  if (!length || !accepted_len || !new_length || !is4(seq) || !is4(length) ||
      !is4(accepted_len) || !is4(path) || !is4(new_length) || extra < 0 || tokens <= 0 ||
      (path && path_width <= 0))
    return DSPARK_ERR_INVALID_ARG;
  if (path && path_width > DSPARK_TREE_MAX_TOKENS) return DSPARK_ERR_UNSUPPORTED;
  return from_cuda(launch_cache_accept(*cache, seq, length, accepted_len, path, path_width,
                                       extra, tokens, B, new_length, stream));
}

dspark_status dspark_cache_append(
    const dspark_cache* cache, int layer, const int32_t* seq, const int32_t* length,
    const int32_t* token_count, const void* q, int64_t q_stride, const void* k,
    int64_t k_stride, const void* v, int64_t v_stride, const float* q_weight,
    const float* k_weight, float eps, const float* cos_sin, int max_position,
    int rot_dim, int interleaved, const int32_t* position, int B, int T, int heads,
    void* q_out, cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st == DSPARK_OK) st = check_heads(heads, cache->kv_heads);
  if (st != DSPARK_OK) return st;
  const int D = cache->head_dim;
  if (!length || !q || !k || !v || !cos_sin || !position || !q_out || T <= 0 || layer < 0 ||
      layer >= cache->layers || max_position <= 0 || rot_dim <= 0 || rot_dim > D ||
      rot_dim % 2 != 0 || !(eps >= 0.0f) || !std::isfinite(eps))
    return DSPARK_ERR_INVALID_ARG;
  const void* p16[] = {q, k, v, q_out};
  for (const void* p : p16)
    if (!aligned_to(p, 16)) return DSPARK_ERR_INVALID_ARG;
  const void* p4[] = {seq, length, token_count, q_weight, k_weight, cos_sin, position};
  for (const void* p : p4)
    if (!is4(p)) return DSPARK_ERR_INVALID_ARG;
  if (q_stride < (int64_t)heads * D || k_stride < (int64_t)cache->kv_heads * D ||
      v_stride < (int64_t)cache->kv_heads * D || q_stride % 8 != 0 || k_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return DSPARK_ERR_INVALID_ARG;
  // q_out may be q only where both lie alike
  if (q_out == q && q_stride != (int64_t)heads * D) return DSPARK_ERR_INVALID_ARG;
  if ((long long)B * T >= (1 << 24) || heads > 32768) return DSPARK_ERR_UNSUPPORTED;
  // warps read rows while others write queries
  const int64_t tokens = (int64_t)B * T, elt = dtype_bytes(cache->dtype);
  const int64_t q_row = heads * D * elt, kv_row = cache->kv_heads * D * elt;
  if ((q_out != q && rows_meet(q, q_stride * (__int128)elt, q_row, tokens, q_out, tokens * q_row)) ||
      rows_meet(k, k_stride * (__int128)elt, kv_row, tokens, q_out, tokens * q_row) ||
      rows_meet(v, v_stride * (__int128)elt, kv_row, tokens, q_out, tokens * q_row))
    return DSPARK_ERR_INVALID_ARG;
  AppendArgs a{};
  a.c = *cache;
  a.layer = layer;
  a.seq = seq;
  a.length = length;
  a.count = token_count;
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_position = max_position;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.position = position;
  a.B = B;
  a.T = T;
  a.heads = heads;
  a.q_out = static_cast<char*>(q_out);
  return from_cuda(launch_cache_append(a, stream));
}

size_t dspark_tree_workspace_bytes(int B, int T, int heads, int kv_heads, int head_dim) {
  if (!tree_sizes(B, T, heads, kv_heads, head_dim)) return 0;
  return tree_layout(T, heads / kv_heads, head_dim).total;
}

dspark_status dspark_tree_attention(
    const dspark_cache* cache, int layer, const int32_t* seq, const int32_t* length,
    const int32_t* token_count, const void* q, const uint64_t* mask, int64_t mask_stride,
    const int32_t* position, int window, float scale, int B, int T, int heads, void* out,
    float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st == DSPARK_OK) st = check_heads(heads, cache->kv_heads);
  if (st != DSPARK_OK) return st;
  if (!length || !q || !out || T <= 0 || layer < 0 || layer >= cache->layers || window < 0 ||
      !std::isfinite(scale) || (mask && mask_stride != 0 && mask_stride < T))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || (mask && !aligned_to(mask, 8)))
    return DSPARK_ERR_INVALID_ARG;
  const void* p4[] = {seq, length, token_count, position, lse};
  for (const void* p : p4)
    if (!is4(p)) return DSPARK_ERR_INVALID_ARG;
  if (!tree_sizes(B, T, heads, cache->kv_heads, cache->head_dim)) return DSPARK_ERR_UNSUPPORTED;
  const int group = heads / cache->kv_heads;
  const TreeLayout L = tree_layout(T, group, cache->head_dim);
  if (!workspace || workspace_bytes < L.total || !aligned_to(workspace, 256))
    return DSPARK_ERR_WORKSPACE;
  // blocks read queries while others write results
  const uintptr_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(out);
  const size_t bytes = (size_t)B * T * heads * cache->head_dim * dtype_bytes(cache->dtype);
  if (from < to + bytes && to < from + bytes) return DSPARK_ERR_INVALID_ARG;
  TreeArgs a{};
  a.c = *cache;
  a.layer = layer;
  a.seq = seq;
  a.length = length;
  a.count = token_count;
  a.position = position;
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.window = window;
  a.scale = scale;
  a.B = B;
  a.T = T;
  a.heads = heads;
  a.group = group;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.join = static_cast<TreeJoin*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.part);
  cudaError_t e = tree_tc_supported(a) ? launch_tree_tc(a, sm_count(), stream)
                                       : launch_tree_ffma(a, sm_count(), stream);
  if (e == cudaSuccess) e = launch_tree_merge(a, stream);
  return from_cuda(e);
}

}  // extern "C"
