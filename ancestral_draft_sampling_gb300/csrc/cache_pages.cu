// cache_pages.cu -- bookkeeping of the paged key/value cache: taking pages
// from the free stack, giving them back, sharing them between sequences, and
// the copies that go with it (the partly filled page of a fork, the rows of
// an accepted path).
//
// The bookkeeping of a call is a few thousand integers, bound by latency: one
// block runs it, with a thread for each sequence and block-wide sums for the
// places on the stack, so the order is fixed and a call needs one launch.
// The copies are bound by HBM and run over the whole GPU.  64 children of four
// parents of 4000 tokens, 16 layers: 9 us of bookkeeping and 29 us of copies,
// 118 MB through HBM; eight wide trees accepted in 10 us, most of it a launch
// and a chain of some ten loads and barriers that depend on each other.
#include <climits>

#include "cache.cuh"
#include "dspark_common.cuh"
#include "host_util.cuh"

namespace dspark {
namespace {

constexpr int kMaxB = DSPARK_CACHE_MAX_B;
constexpr int kBlock = 1024;  // threads of a bookkeeping block

// The entries of the block table that a call gives up: of row b those from
// from[b] on, offset[b + 1] - offset[b] of them.
struct GiveList {
  int seq[kMaxB];
  int from[kMaxB];
  int offset[kMaxB + 1];
};

// The row of flat entry e.
__device__ __forceinline__ int row_of(const int* offset, int B, int e) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offset[mid] <= e) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// offset[] from each row's count (thread b holds row b's; B <= blockDim
// passes of blockDim rows otherwise).
__device__ __forceinline__ void row_offsets(int* offset, const int* counts,
                                            int B, int* warps) {
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const int n = b < B ? counts[b] : 0;
    int total;
    const int x = block_exclusive(n, warps, total);
    if (b < B) offset[b] = base + x;
    base += total;
  }
  if (threadIdx.x == 0) offset[B] = base;
  __syncthreads();
}

// The same for a list of any length: the entries are walked anew in each step.
__device__ __noinline__ int give_many(const dspark_cache& c, const GiveList& g, int B, int top,
                                      int* warps) {
  const int n = g.offset[B];
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int b = row_of(g.offset, B, e);
    const int i = g.from[b] + e - g.offset[b];
    const int p = cache_page(c, g.seq[b], i, c.max_pages);
    if (p >= 0) atomicSub(&c.ref_count[p], 1);
    else cache_error(c, kCacheErrPage);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int b = row_of(g.offset, B, e);
    const int p = cache_page(c, g.seq[b], g.from[b] + e - g.offset[b], c.max_pages);
    if (p >= 0 && __ldcg(&c.ref_count[p]) <= 0)
      atomicMin(&c.ref_count[p], INT_MIN + e);
  }
  __syncthreads();
  for (int e0 = 0; e0 < n; e0 += blockDim.x) {
    const int e = n - 1 - e0 - (int)threadIdx.x;  // from the last entry on
    int p = -1;
    if (e >= 0) {
      const int b = row_of(g.offset, B, e);
      p = c.block_table[(size_t)g.seq[b] * c.max_pages + g.from[b] + e - g.offset[b]];
      if (p < 0 || p >= c.num_pages || __ldcg(&c.ref_count[p]) != INT_MIN + e) p = -1;
    }
    int total;
    const int x = block_exclusive(p >= 0, warps, total);
    if (p >= 0) {
      __stcg(&c.ref_count[p], 0);
      if (top + x >= 0 && top + x < c.num_pages) c.free_list[top + x] = p;
    }
    top += total;
  }
  for (int e = threadIdx.x; e < n; e += blockDim.x) {  // a row may be listed twice
    const int b = row_of(g.offset, B, e);
    c.block_table[(size_t)g.seq[b] * c.max_pages + g.from[b] + e - g.offset[b]] = -1;
  }
  return top;
}

// Takes one hold off each listed page; the pages that nobody holds any more
// go on the free stack, the last listed first.  A page that is listed several
// times goes there once, for its first entry: after the holds are taken off,
// the entries of a page without holds compete with an atomic minimum over
// their numbers, in the page's own count (the order does not matter to a
// minimum, so the stack is the same on every run).  There is nothing to
// compete for where each page either had one hold or still has some, and no
// places to count where all go on the stack.
// Up to four entries a thread are walked once and held in registers (4096
// entries: 13 us with the launch, where the general form takes 22); longer lists
// take the general form, a chain of four walks in one block: 4160 entries 25 us,
// 22000 pages of 88 sequences 84 us.  A sequence gives up so many pages once.
constexpr int kPer = 4;  // entries of a thread, their loads in flight together

__device__ void give_pages(const dspark_cache& c, const GiveList& g, int B,
                           int* warps) {
  const int n = g.offset[B], before = c.control[kCtlFree];
  int top = before;
  if (n > kPer * (int)blockDim.x) {
    top = give_many(c, g, B, before, warps);
  } else {
    int page[kPer], held[kPer];
    size_t at[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = threadIdx.x + k * blockDim.x;
      page[k] = -1;
      held[k] = 1;
      if (e >= n) continue;
      const int b = row_of(g.offset, B, e);
      at[k] = (size_t)g.seq[b] * c.max_pages + g.from[b] + e - g.offset[b];
      page[k] = c.block_table[at[k]];
    }
    __syncthreads();  // a row may be listed twice
    bool plain = true;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (threadIdx.x + k * blockDim.x >= n) continue;
      if (page[k] >= 0 && page[k] < c.num_pages) {
        held[k] = atomicSub(&c.ref_count[page[k]], 1);
      } else {
        page[k] = -1;
        cache_error(c, kCacheErrPage);
      }
      c.block_table[at[k]] = -1;
      plain &= page[k] >= 0 && held[k] == 1;
    }
    if (__syncthreads_and(plain)) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int to = top + n - 1 - (int)(threadIdx.x + k * blockDim.x);
        if (page[k] >= 0 && to >= 0 && to < c.num_pages) c.free_list[to] = page[k];
      }
      top += n;
    } else {
      bool compete = false;
      int left[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        left[k] = page[k] >= 0 ? __ldcg(&c.ref_count[page[k]]) : 1;
        compete |= page[k] >= 0 && held[k] != 1 && left[k] <= 0;
      }
      compete = __syncthreads_or(compete);
      if (compete) {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (left[k] <= 0)
            atomicMin(&c.ref_count[page[k]], INT_MIN + (int)(threadIdx.x + k * blockDim.x));
        __syncthreads();
      }
      int place[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = threadIdx.x + k * blockDim.x;
        const bool goes = left[k] <= 0 &&
                          (!compete || __ldcg(&c.ref_count[page[k]]) == INT_MIN + e);
        int total;
        place[k] = top + block_exclusive(goes, warps, total);
        if (!goes) page[k] = -1;
        top += total;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int to = before + top - 1 - place[k];
        if (page[k] < 0) continue;
        __stcg(&c.ref_count[page[k]], 0);
        if (to >= 0 && to < c.num_pages) c.free_list[to] = page[k];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) c.control[kCtlFree] = top < c.num_pages ? top : c.num_pages;
  for (int b = threadIdx.x; b < B; b += blockDim.x)
    if (g.offset[b + 1] > g.offset[b]) c.page_count[g.seq[b]] = g.from[b];
  __syncthreads();
}

// How many of each row's wanted pages it gets, in the rows' order: all of
// them, or, where the stack runs out, none for the rows that do not fit.
// need[b] becomes what row b gets.
__device__ __forceinline__ void grant(const dspark_cache& c, int* need, int* offset,
                                      int B, int free, int* warps) {
  row_offsets(offset, need, B, warps);
  if (offset[B] > free) {
    if (threadIdx.x == 0) {
      int left = free;
      for (int b = 0; b < B; ++b) {
        if (need[b] > left) {
          need[b] = 0;
          cache_error(c, kCacheErrFull);
        }
        left -= need[b];
      }
    }
    __syncthreads();
    row_offsets(offset, need, B, warps);
  }
}

__device__ __forceinline__ int free_pages(const dspark_cache& c) {
  const int n = c.control[kCtlFree];
  return n < 0 ? 0 : n > c.num_pages ? c.num_pages : n;
}

__global__ void init_kernel(dspark_cache c) {
  follow();
  const size_t n = (size_t)gridDim.x * blockDim.x;
  const size_t i0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (size_t i = i0; i < (size_t)c.max_seqs * c.max_pages; i += n) c.block_table[i] = -1;
  for (size_t i = i0; i < (size_t)c.max_seqs; i += n) c.page_count[i] = 0;
  for (size_t i = i0; i < (size_t)c.num_pages; i += n) {
    c.ref_count[i] = 0;
    c.free_list[i] = c.num_pages - 1 - (int)i;
  }
  if (i0 < 64) c.control[i0] = i0 == kCtlFree ? c.num_pages : 0;
}

__global__ void __launch_bounds__(kBlock, 1)
    reserve_kernel(dspark_cache c, const int32_t* seq, const int32_t* length,
                   int tokens, int B) {
  __shared__ int need[kMaxB], have[kMaxB], seqs[kMaxB], offset[kMaxB + 1], warps[33];
  const int b = threadIdx.x;
  follow();
  if (b < B) {
    const int s = cache_seq(c, seq, b), len = length[b];
    int n = 0, h = 0;
    if (s < 0) {
      cache_error(c, kCacheErrSeq);
    } else if (len < 0) {
      cache_error(c, kCacheErrPage);
    } else {
      h = cache_held(c, s);
      const uint32_t want = pages_for(c, (uint32_t)len + (uint32_t)tokens);
      if (want > (uint32_t)c.max_pages) cache_error(c, kCacheErrFull);
      else if ((int)want > h) n = (int)want - h;
    }
    need[b] = n;
    have[b] = h;
    seqs[b] = s;
  }
  __syncthreads();
  const int free = free_pages(c);
  grant(c, need, offset, B, free, warps);
  const int total = offset[B];
  for (int e = threadIdx.x; e < total; e += blockDim.x) {
    const int r = row_of(offset, B, e);
    const int p = c.free_list[free - 1 - e];
    c.block_table[(size_t)seqs[r] * c.max_pages + have[r] + e - offset[r]] = p;
    if (p >= 0 && p < c.num_pages) c.ref_count[p] = 1;
    else cache_error(c, kCacheErrPage);
  }
  if (b < B && need[b] > 0) c.page_count[seqs[b]] = have[b] + need[b];
  if (threadIdx.x == 0 && total > 0) c.control[kCtlFree] = free - total;
}

__global__ void __launch_bounds__(kBlock, 1)
    release_kernel(const __grid_constant__ dspark_cache c, const int32_t* seq, int B) {
  __shared__ GiveList g;
  __shared__ int counts[kMaxB], warps[33];
  const int b = threadIdx.x;
  follow();
  if (b < B) {
    const int s = cache_seq(c, seq, b);
    if (s < 0) cache_error(c, kCacheErrSeq);
    g.seq[b] = s;
    g.from[b] = 0;
    counts[b] = s < 0 ? 0 : cache_held(c, s);
  }
  __syncthreads();
  row_offsets(g.offset, counts, B, warps);
  give_pages(c, g, B, warps);
}

// Fork, the bookkeeping: gives up the children's pages and takes a page for
// each partly filled one.  Scratch words 2 b and 2 b + 1 tell the copy what to
// do: how many of the parent's pages to share, and the page to copy the next
// one's rows to, or -1.
__global__ void __launch_bounds__(kBlock, 1)
    fork_kernel(const __grid_constant__ dspark_cache c, const int32_t* parent, const int32_t* child,
                const int32_t* length, int B) {
  __shared__ GiveList g;
  __shared__ int par[kMaxB], full[kMaxB], need[kMaxB], warps[33];
  int* scratch = c.control + kCtlScratch;
  const int b = threadIdx.x;
  follow();
  int len = 0, p = -1, s = -1;
  if (b < B) {
    p = cache_seq(c, parent, b);
    s = cache_seq(c, child, b);
    len = length[b];
    scratch[2 * b] = 0;
    scratch[2 * b + 1] = -1;
    if (p < 0 || s < 0) {
      cache_error(c, kCacheErrSeq);
      s = -1;
    }
    par[b] = p;
    g.seq[b] = s;
  }
  __syncthreads();
  bool clash = false;
  if (b < B && s >= 0)
    for (int i = 0; i < B; ++i)
      clash |= par[i] == s || (i != b && g.seq[i] == s);
  if (__syncthreads_or(clash)) {  // the whole call does nothing
    if (threadIdx.x == 0) cache_error(c, kCacheErrFork);
    return;
  }
  if (b < B) {
    g.from[b] = 0;
    need[b] = s < 0 ? 0 : cache_held(c, s);
  }
  __syncthreads();
  row_offsets(g.offset, need, B, warps);
  give_pages(c, g, B, warps);
  if (b < B) {
    int f = 0, n = 0;
    if (s >= 0) {
      if (len < 0 || len > cache_held(c, p) * c.page_size) {  // at most 2^30
        cache_error(c, kCacheErrPage);
      } else {
        int rest;
        f = (int)page_of(c, (uint32_t)len, rest);
        n = rest > 0 ? 1 : 0;
      }
    }
    full[b] = f;
    need[b] = n;
  }
  const bool partly = b < B && need[b] > 0;
  __syncthreads();
  const int free = free_pages(c);
  int* offset = g.offset;
  grant(c, need, offset, B, free, warps);
  const int taken = offset[B];
  if (b < B && s >= 0) {
    if (partly && need[b] == 0) full[b] = 0;  // no page left: the child is empty
    if (need[b] > 0) {
      const int to = c.free_list[free - 1 - offset[b]];
      const int from = cache_page(c, p, full[b], c.max_pages);
      c.block_table[(size_t)s * c.max_pages + full[b]] = to;
      if (to >= 0 && to < c.num_pages) {
        c.ref_count[to] = 1;
        scratch[2 * b + 1] = from >= 0 ? to : -1;
      }
      if (from < 0 || to < 0 || to >= c.num_pages) cache_error(c, kCacheErrPage);
    }
    c.page_count[s] = full[b] + need[b];
    scratch[2 * b] = full[b];
  }
  if (threadIdx.x == 0 && taken > 0) c.control[kCtlFree] = free - taken;
}

// Fork, the rest: the first block of child b shares the parent's full pages (in
// the bookkeeping's one block, 4000 entries take 4 us), and a warp for each (plane, head) of child b copies the filled
// rows, which are contiguous there, eight 16-byte words a lane in flight.
// Bound by HBM: each child's rows are written once; they are read from L2 when
// several children share a parent.
constexpr int kCopyThreads = 256, kCopyBatch = 8;

__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(dspark_cache c, const int32_t* parent, const int32_t* child,
                     const int32_t* length) {
  follow();
  const int b = blockIdx.y;
  const int full = __ldcg(&c.control[kCtlScratch + 2 * b]);
  const int to = __ldcg(&c.control[kCtlScratch + 2 * b + 1]);
  const int p = cache_seq(c, parent, b), s = cache_seq(c, child, b);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < full; i += kCopyThreads) {
      const int id = cache_page(c, p, i, c.max_pages);
      c.block_table[(size_t)s * c.max_pages + i] = id;
      if (id >= 0) atomicAdd(&c.ref_count[id], 1);
      else cache_error(c, kCacheErrPage);
    }
  }
  if (to < 0) return;
  const int from = cache_page(c, p, full, c.max_pages);
  int rows;
  page_of(c, (uint32_t)length[b], rows);
  const int words = rows * (c.head_dim * dtype_bytes(c.dtype) / 16);
  const int lane = threadIdx.x & 31, items = 2 * c.layers * c.kv_heads;
  char* pool = static_cast<char*>(c.pool);
  for (int item = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); item < items;
       item += gridDim.x * (kCopyThreads / 32)) {
    const int plane = item / c.kv_heads, head = item - plane * c.kv_heads;
    const uint4* src = reinterpret_cast<const uint4*>(pool + cache_row(c, plane, from, head, 0));
    uint4* dst = reinterpret_cast<uint4*>(pool + cache_row(c, plane, to, head, 0));
    for (int i = lane; i < words; i += 32 * kCopyBatch) {
      uint4 v[kCopyBatch];
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k)
        if (i + 32 * k < words) v[k] = src[i + 32 * k];
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k)
        if (i + 32 * k < words) dst[i + 32 * k] = v[k];
    }
  }
}

// Accept.  Block (x, b) moves its share of the rows of sequence b; block
// (0, b) leaves the number of kept tokens in the scratch.  The block that
// finishes last (a ticket; nobody waits) writes the new lengths and gives up
// the pages behind them.  The rows of a path are moved in order by one thread
// for each 16-byte column of a (plane, head): path[i] increases strictly from
// path[0] >= 0, so path[i] >= i and a row is read before any later row lands
// on it; eight rows are loaded before the first is stored, and none of the
// eight destinations i .. i + 7 is a source behind them (path[i + 8] > i + 7).
constexpr int kMoveThreads = 256, kMoveBatch = 8;

__global__ void __launch_bounds__(kMoveThreads)
    accept_kernel(const __grid_constant__ dspark_cache c, const int32_t* seq, const int32_t* length,
                  const int32_t* accepted, const int32_t* path, int path_width,
                  int extra, int tokens, int B, int32_t* new_length) {
  __shared__ GiveList g;
  __shared__ int counts[kMaxB], warps[33];
  __shared__ size_t src[DSPARK_TREE_MAX_TOKENS], dst[DSPARK_TREE_MAX_TOKENS];
  __shared__ int first_move, last_block;
  int* scratch = c.control + kCtlScratch;
  const int b = blockIdx.y;
  follow();
  const int s = cache_seq(c, seq, b), len = length[b], acc = accepted[b];
  const uint32_t wanted = acc < 0 ? 0u : (uint32_t)acc + (uint32_t)extra;
  const int most = path ? path_width : tokens;
  const int held = s < 0 ? 0 : cache_held(c, s);
  int err = s < 0 ? kCacheErrSeq : 0;
  if (!err && (wanted > (uint32_t)most || wanted > (uint32_t)tokens)) err = kCacheErrPath;
  if (!err && (len < 0 || (uint32_t)len + wanted > (uint32_t)(held * c.page_size)))
    err = kCacheErrPage;  // both below 2^31; held pages hold at most 2^30
  int n = err ? 0 : (int)wanted;
  if (threadIdx.x == 0) first_move = DSPARK_TREE_MAX_TOKENS;
  __syncthreads();
  if (path) {  // n <= path_width <= DSPARK_TREE_MAX_TOKENS
    bool bad = false, unheld = false;
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
      const int at = path[(size_t)b * path_width + i];
      const int before = i > 0 ? path[(size_t)b * path_width + i - 1] : -1;
      if (at <= before || at >= tokens) {
        bad = true;
        continue;
      }
      int from_slot, to_slot;
      const uint32_t fi = page_of(c, (uint32_t)len + (uint32_t)at, from_slot);
      const int from = fi < (uint32_t)held ? cache_page(c, s, (int)fi, held) : -1;
      const int to = cache_page(c, s, (int)page_of(c, (uint32_t)(len + i), to_slot), held);
      if (from < 0 || to < 0) {
        unheld = true;
        continue;
      }
      src[i] = cache_row(c, 0, from, 0, from_slot);
      dst[i] = cache_row(c, 0, to, 0, to_slot);
      if (at != i) atomicMin(&first_move, i);
    }
    if (__syncthreads_or(bad)) err = kCacheErrPath;
    else if (__syncthreads_or(unheld)) err = kCacheErrPage;
    if (err) n = 0;
    const int words = c.head_dim * dtype_bytes(c.dtype) / 16;
    const size_t head_step = cache_row(c, 0, 0, 1, 0), plane_step = cache_row(c, 1, 0, 0, 0);
    const unsigned columns = 2u * c.layers * c.kv_heads * words;
    char* pool = static_cast<char*>(c.pool);
    for (unsigned i = blockIdx.x * kMoveThreads + threadIdx.x; i < columns && first_move < n;
         i += gridDim.x * kMoveThreads) {
      const unsigned item = i / words, plane = item / c.kv_heads, head = item % c.kv_heads;
      char* at = pool + plane * plane_step + head * head_step + 16 * (size_t)(i % words);
      for (int r = first_move; r < n; r += kMoveBatch) {
        uint4 v[kMoveBatch];
#pragma unroll
        for (int k = 0; k < kMoveBatch; ++k)
          if (r + k < n) v[k] = *reinterpret_cast<const uint4*>(at + src[r + k]);
#pragma unroll
        for (int k = 0; k < kMoveBatch; ++k)
          if (r + k < n) *reinterpret_cast<uint4*>(at + dst[r + k]) = v[k];
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    scratch[b] = n;
    if (err) cache_error(c, err);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int all = gridDim.x * gridDim.y;
    last_block = atomicAdd(&c.control[kCtlTicket], 1) == all - 1;
    if (last_block) c.control[kCtlTicket] = 0;
  }
  __syncthreads();
  if (!last_block) return;
  __threadfence();
  for (int i = threadIdx.x; i < B; i += kMoveThreads) {
    const int si = cache_seq(c, seq, i);
    const int now = length[i] + __ldcg(&scratch[i]);
    int from = 0, count = 0;
    if (si >= 0 && now >= 0) {
      const int h = cache_held(c, si);
      from = (int)pages_for(c, (uint32_t)now);
      count = h > from ? h - from : 0;
    }
    g.seq[i] = si;
    g.from[i] = from;
    counts[i] = count;
    new_length[i] = now;
  }
  __syncthreads();
  row_offsets(g.offset, counts, B, warps);
  if (g.offset[B] > 0) give_pages(c, g, B, warps);
}

}  // namespace

// Threads for B sequences and the pages that they may hold: a block-wide step
// of few warps is shorter.
static int list_threads(const dspark_cache& c, int B) {
  const long long most = (long long)B * c.max_pages;
  return B <= 128 && most <= 128 * kPer ? 128 : kBlock;
}

cudaError_t launch_cache_init(const dspark_cache& c, cudaStream_t stream) {
  const size_t most = (size_t)c.max_seqs * c.max_pages > (size_t)c.num_pages
                          ? (size_t)c.max_seqs * c.max_pages
                          : (size_t)c.num_pages;
  const size_t blocks = (most + 255) / 256;
  return launch_behind(init_kernel, (unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, stream, c);
}

cudaError_t launch_cache_reserve(const dspark_cache& c, const int32_t* seq,
                                 const int32_t* length, int tokens, int B,
                                 cudaStream_t stream) {
  // a thread for each sequence: fewer warps to sum over where there are few
  const int threads = B <= 128 ? 128 : kBlock;
  return launch_behind(reserve_kernel, 1, threads, 0, stream, c, seq, length, tokens, B);
}

cudaError_t launch_cache_release(const dspark_cache& c, const int32_t* seq,
                                 int B, cudaStream_t stream) {
  return launch_behind(release_kernel, 1, list_threads(c, B), 0, stream, c, seq, B);
}

cudaError_t launch_cache_fork(const dspark_cache& c, const int32_t* parent,
                              const int32_t* child, const int32_t* length,
                              int B, cudaStream_t stream) {
  cudaError_t e = launch_behind(fork_kernel, 1, list_threads(c, B), 0, stream, c, parent, child,
                                length, B);
  if (e != cudaSuccess) return e;
  const int items = 2 * c.layers * c.kv_heads;
  const int blocks = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return launch_behind(fork_copy_kernel, dim3(blocks, B), kCopyThreads, 0, stream, c, parent,
                       child, length);
}

cudaError_t launch_cache_accept(const dspark_cache& c, const int32_t* seq,
                                const int32_t* length, const int32_t* accepted,
                                const int32_t* path, int path_width, int extra,
                                int tokens, int B, int32_t* new_length,
                                cudaStream_t stream) {
  unsigned x = 1;
  if (path) {
    const size_t columns = cache_row(c, 0, 0, 1, 0) / c.page_size / 16 * 2 *
                           c.layers * c.kv_heads;
    const size_t blocks = (columns + kMoveThreads - 1) / kMoveThreads;
    x = (unsigned)(blocks < 1024 ? blocks : 1024);
  }
  return launch_behind(accept_kernel, dim3(x, B), kMoveThreads, 0, stream, c, seq, length,
                       accepted, path, path_width, extra, tokens, B, new_length);
}

}  // namespace dspark
