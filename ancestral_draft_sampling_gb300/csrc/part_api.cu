// part_api.cu -- the C ABI of what reads part of the cache (include/dspark.h):
// bounds of pages, their selection, the attention over selected pages and that
// over shared prefixes.
#include <cmath>

#include "cache_check.cuh"
#include "part_attention.cuh"
#include "select_pages.cuh"

namespace {

using namespace dspark;

size_t align_up(size_t x, size_t n) { return (x + n - 1) / n * n; }

// The workspace of the selection: the scores of every list, the exact ones of
// many pages near the border, and what bounds the scores' errors.
struct SelectLayout {
  int stride, reaches;
  size_t border, reach_q, reach_k, total;
};

SelectLayout select_layout(const dspark_cache& c, int B, int T, int lists) {
  SelectLayout L;
  L.stride = (c.max_pages + 3) / 4 * 4;
  L.reaches = (c.max_pages + 15) / 16 * 16 / kReachPages;  // of whole warps' 16 pages
  const size_t rows = (size_t)B * lists * c.kv_heads;
  L.border = align_up(rows * L.stride * sizeof(float), 256);
  L.reach_q = align_up(L.border + rows * L.stride * sizeof(uint64_t), 256);
  L.reach_k = align_up(L.reach_q + (size_t)B * T * c.kv_heads * sizeof(float), 256);
  L.total = align_up(L.reach_k + (size_t)B * c.kv_heads * L.reaches * sizeof(float), 256);
  return L;
}

dspark_status select_sizes(const dspark_cache* c, int B, int T) {
  if (B <= 0 || T <= 0) return DSPARK_ERR_INVALID_ARG;
  // stretches of tables are counted in 32 bits
  if (B > DSPARK_CACHE_MAX_B || T > DSPARK_TREE_MAX_TOKENS ||
      (long long)B * c->kv_heads * ((c->max_pages + 63) / 64) >= (1LL << 31))
    return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

// The checks of the attention's sizes.
dspark_status attention_sizes(int B, int T, int heads, int kv_heads, int D) {
  if (B <= 0 || T <= 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0) return DSPARK_ERR_INVALID_ARG;
  if (B > DSPARK_CACHE_MAX_B || T > DSPARK_TREE_MAX_TOKENS || kv_heads > 1024 ||
      heads / kv_heads > DSPARK_TREE_MAX_GROUP || D < 8 || D > 256 || D % 8 != 0)
    return DSPARK_ERR_UNSUPPORTED;
  return DSPARK_OK;
}

dspark_status prefix_sizes(int B, int T, int heads, int kv_heads, int D) {
  const dspark_status st = attention_sizes(B, T, heads, kv_heads, D);
  // rows of results are counted in 32 bits
  return st == DSPARK_OK && (long long)B * T * heads >= (1LL << 31) ? DSPARK_ERR_UNSUPPORTED : st;
}

// What the attention needs for units of up to `tokens` tokens, `items` of them:
// the merge's work, partial results (two a block), the items and their work.
struct ItemLayout {
  size_t part, items, work, end;
};

ItemLayout item_layout(long long tokens, size_t items, int group, int D) {
  ItemLayout L;
  L.part = align_up((size_t)2 * kTreeMaxBlocks * sizeof(TreeJoin), 256);
  const int fit = 2 * (kTreeRows / group);  // tokens of a tensor-core unit, the largest
  const size_t rows = (size_t)(tokens < fit ? tokens : fit) * group * 2 * kTreeMaxBlocks;
  L.items = align_up(L.part + rows * (D + 2) * sizeof(float), 256);
  L.work = align_up(L.items + items * sizeof(TreeItem), 256);
  L.end = align_up(L.work + items * sizeof(long long), 256);
  return L;
}

struct SparseLayout {
  ItemLayout items;
  int room;
  size_t list, bits, total;
};

SparseLayout sparse_layout(const dspark_cache& c, int B, int T, int heads, int count) {
  SparseLayout L;
  const size_t n = (size_t)B * c.kv_heads;
  L.items = item_layout(T, n, heads / c.kv_heads, c.head_dim);
  const long long named = (long long)count * T;
  L.room = (int)(named < c.max_pages ? named : c.max_pages) + T / c.page_size + 2;
  L.list = L.items.end;
  L.bits = align_up(L.list + n * L.room * sizeof(int32_t), 256);
  L.total = align_up(L.bits + n * L.room * sizeof(uint64_t), 256);
  return L;
}

struct PrefixLayout {
  ItemLayout shared, own;
  size_t base, group_of, whole, total;
};

PrefixLayout prefix_layout(int B, int T, int heads, int kv_heads, int D) {
  PrefixLayout L;
  const int group = heads / kv_heads;
  L.shared = item_layout((long long)B * T, (size_t)2 * B, group, D);
  L.own = item_layout(T, B, group, D);  // behind it
  L.base = L.shared.end + L.own.end;
  L.group_of = align_up(L.base + ((size_t)2 * B + 4) * sizeof(long long), 256);
  L.whole = align_up(L.group_of + (size_t)B * sizeof(int32_t), 256);
  L.total = align_up(L.whole + (size_t)2 * B * T * heads * (D + 2) * sizeof(float), 256);
  return L;
}

// What both attentions check, and the arguments that they share.
dspark_status fill_attention(TreeArgs& a, const dspark_cache* cache, int layer, const int32_t* seq,
                             const int32_t* length, const int32_t* token_count, const void* q,
                             const uint64_t* mask, int64_t mask_stride, float scale, int B, int T,
                             int heads, void* out, float* lse) {
  dspark_status st = check_cache(cache);
  if (st == DSPARK_OK) st = check_batch(B);
  if (st == DSPARK_OK) st = check_heads(heads, cache->kv_heads);
  if (st != DSPARK_OK) return st;
  if (!length || !q || !out || T <= 0 || layer < 0 || layer >= cache->layers ||
      !std::isfinite(scale) || (mask && mask_stride != 0 && mask_stride < T))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || (mask && !aligned_to(mask, 8)))
    return DSPARK_ERR_INVALID_ARG;
  const void* p4[] = {seq, length, token_count, lse};
  for (const void* p : p4)
    if (!is4(p)) return DSPARK_ERR_INVALID_ARG;
  st = attention_sizes(B, T, heads, cache->kv_heads, cache->head_dim);
  if (st != DSPARK_OK) return st;
  // blocks read queries while others write results
  const uintptr_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(out);
  const size_t bytes = (size_t)B * T * heads * cache->head_dim * dtype_bytes(cache->dtype);
  if (from < to + bytes && to < from + bytes) return DSPARK_ERR_INVALID_ARG;
  a.c = *cache;
  a.layer = layer;
  a.seq = seq;
  a.length = length;
  a.count = token_count;
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.scale = scale;
  a.B = B;
  a.T = T;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.q = q;
  a.out = out;
  a.lse = lse;
  return DSPARK_OK;
}

void fill_items(TreeArgs& a, const ItemLayout& L, char* ws) {
  a.join = reinterpret_cast<TreeJoin*>(ws);
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.items = reinterpret_cast<TreeItem*>(ws + L.items);
  a.item_work = reinterpret_cast<long long*>(ws + L.work);
}

void plan(TreeArgs& a, int tokens) {
  if (items_tc_supported(a)) {
    tree_tc_plan(a, tokens, sm_count());
    // in tiles: 4000 cycles of a narrow unit's end, of 1425 a tile of 64 dims and 2850
    // of 128; 8000 of 3470 for a pair of tiles of 256 rows
    a.extra = !tree_tc_narrow(a, tokens) ? 2 : a.c.head_dim <= 64 ? 3 : 1;
  } else {
    tree_ffma_plan(a, tokens, sm_count());
  }
}

cudaError_t launch_items(const TreeArgs& a, cudaStream_t stream) {
  return items_tc_supported(a) ? launch_items_tc(a, stream) : launch_items_ffma(a, stream);
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
  return select_layout(*cache, B, T, shared ? 1 : T).total;
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
  const SelectLayout L = select_layout(*cache, B, T, lists);
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
  a.reaches = L.reaches;
  char* ws = static_cast<char*>(workspace);
  a.scores = reinterpret_cast<float*>(ws);
  a.border = reinterpret_cast<uint64_t*>(ws + L.border);
  a.reach_q = reinterpret_cast<float*>(ws + L.reach_q);
  a.reach_k = reinterpret_cast<float*>(ws + L.reach_k);
  return from_cuda(launch_select_pages(a, sm_count(), stream));
}

size_t dspark_sparse_workspace_bytes(const dspark_cache* cache, int B, int T, int heads, int count) {
  if (check_cache(cache) != DSPARK_OK || count <= 0 || (long long)count * T > (1 << 24) ||
      attention_sizes(B, T, heads, cache->kv_heads, cache->head_dim) != DSPARK_OK)
    return 0;
  return sparse_layout(*cache, B, T, heads, count).total;
}

dspark_status dspark_sparse_attention(const dspark_cache* cache, int layer, const int32_t* seq,
                                      const int32_t* length, const int32_t* token_count, const void* q,
                                      const int32_t* pages, int count, int shared, const uint64_t* mask,
                                      int64_t mask_stride, float scale, int B, int T, int heads,
                                      void* out, float* lse, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
  SparseArgs p{};
  const dspark_status st = fill_attention(p.a, cache, layer, seq, length, token_count, q, mask,
                                          mask_stride, scale, B, T, heads, out, lse);
  if (st != DSPARK_OK) return st;
  if (!pages || !is4(pages) || count <= 0) return DSPARK_ERR_INVALID_ARG;
  if ((long long)count * T > (1 << 24)) return DSPARK_ERR_UNSUPPORTED;
  const SparseLayout L = sparse_layout(*cache, B, T, heads, count);
  if (!workspace || workspace_bytes < L.total || !aligned_to(workspace, 256))
    return DSPARK_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  fill_items(p.a, L.items, ws);
  p.a.item_count = B * cache->kv_heads;
  p.a.page_list = reinterpret_cast<int32_t*>(ws + L.list);
  p.a.page_bits = reinterpret_cast<uint64_t*>(ws + L.bits);
  p.pages = pages;
  p.count = count;
  p.lists = shared ? 1 : T;
  p.room = L.room;
  plan(p.a, T);
  cudaError_t e = launch_sparse_items(p, stream);
  if (e == cudaSuccess) e = launch_items(p.a, stream);
  if (e == cudaSuccess) e = launch_tree_merge(p.a, stream);
  return from_cuda(e);
}

size_t dspark_prefix_workspace_bytes(int B, int T, int heads, int kv_heads, int head_dim) {
  if (prefix_sizes(B, T, heads, kv_heads, head_dim) != DSPARK_OK) return 0;
  return prefix_layout(B, T, heads, kv_heads, head_dim).total;
}

dspark_status dspark_prefix_attention(const dspark_cache* cache, int layer, const int32_t* seq,
                                      const int32_t* length, const int32_t* token_count, const void* q,
                                      const int32_t* group_start, const int32_t* prefix, int groups,
                                      const uint64_t* mask, int64_t mask_stride, float scale, int B,
                                      int T, int heads, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  PrefixArgs p{};
  TreeArgs& a = p.shared;
  dspark_status st = fill_attention(a, cache, layer, seq, length, token_count, q, mask,
                                    mask_stride, scale, B, T, heads, out, lse);
  if (st != DSPARK_OK) return st;
  if (!group_start || !prefix || !is4(group_start) || !is4(prefix) || groups <= 0 || groups > B)
    return DSPARK_ERR_INVALID_ARG;
  st = prefix_sizes(B, T, heads, cache->kv_heads, cache->head_dim);
  if (st != DSPARK_OK) return st;
  const PrefixLayout L = prefix_layout(B, T, heads, cache->kv_heads, cache->head_dim);
  if (!workspace || workspace_bytes < L.total || !aligned_to(workspace, 256))
    return DSPARK_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  fill_items(a, L.shared, ws);
  a.item_base = reinterpret_cast<long long*>(ws + L.base);
  a.page_list = cache->block_table;
  a.whole = reinterpret_cast<float*>(ws + L.whole);
  p.group_start = group_start;
  p.prefix = prefix;
  p.groups = groups;
  p.group_of = reinterpret_cast<int32_t*>(ws + L.group_of);
  // A sequence's rows are few, a group's many: where that makes different forms of the
  // tensor-core kernel, each kind is launched in its own.  88 single tokens of 8 heads
  // behind a prefix of 4000 keys: one line in the form of many rows 119 us, a launch for
  // each kind 92; 64 x 8 tokens, 16 behind each of four prefixes of up to 16000 keys: 139
  // and 136.  (One launch whose blocks are shared out between both kinds: 99 and 159 us,
  // with blocks that others' loads delay.)
  p.two = items_tc_supported(a) && tree_tc_narrow(a, T) && !tree_tc_narrow(a, B * T);
  p.own = a;
  plan(a, B * T);
  a.item_count = p.two ? groups : groups + B;
  if (p.two) {
    fill_items(p.own, L.own, ws + L.shared.end);
    p.own.item_base = a.item_base + groups + 2;
    p.own.item_count = B;
    plan(p.own, T);
  }
  cudaError_t e = launch_prefix_items(p, stream);
  if (e == cudaSuccess) e = launch_items(a, stream);
  if (e == cudaSuccess && p.two) e = launch_items(p.own, stream);
  if (e == cudaSuccess) e = launch_prefix_join(p, stream);
  return from_cuda(e);
}

}  // extern "C"
