// tree_attention.cuh -- what the kernels of the attention over the paged
// cache share: the work of a call as one line of key tiles, and each block's
// share of it.
//
// A unit is (sequence b, key head h, row tile): up to `row_tokens` drafted
// tokens with their `group` query heads each, row r = (token - first) * group
// + head, over the sequence's keys in tiles of `tile`.  All units' tiles, in
// the order b, h, row tile, form one line of W tiles, and block c of G takes
// tiles c W / G .. (c + 1) W / G: equal shares whatever the lengths.  A unit
// whose tiles lie in one block is finished there; the others leave partial
// results (unnormalised sums, the maximum and the sum of each row), at most
// two a block (its first and its last unit), which the merge kernel joins in
// the blocks' order, so results do not depend on timing.  Only G - 1 places of
// the line can lie inside a unit, so block c of the merge looks after the unit
// that the start of share c cuts first, which block c describes to it (a merge
// block for each unit, each finding its own parts, took 45 us of 150 for 256
// units of 128 rows).
#pragma once

#include "cache.cuh"

namespace dspark {

// Partial results to join: those of blocks first .. last (first's in `slot`,
// the others' in their slot 0) of drafted tokens t0 .. t0 + rows / group - 1.
// rows = 0: nothing.
struct TreeJoin {
  int b, h, t0, rows;
  int first, last, slot, unused;
};

struct TreeArgs {
  dspark_cache c;
  int layer;
  const int32_t *seq, *length, *count, *position;
  const uint64_t* mask;
  long long mask_stride;
  int window;
  float scale;
  int B, T, heads, group;
  const void* q;
  void* out;
  float* lse;
  // schedule
  int blocks;      // G
  int tile;        // keys of a tile
  int row_tokens;  // drafted tokens of a row tile
  int row_tiles;   // of T tokens
  int slot_rows;   // rows of a partial result
  float stat_log2, stat_ln;  // a partial maximum's unit in log2 and in ln units
  struct TreeJoin* join;  // [G] what block c of the merge has to do
  float* part;        // [2 G][slot_rows][D] sums, then [2 G][slot_rows][2]
};

constexpr int kTreeMaxBlocks = 160;   // blocks of a call (the GPU has 152 SMs)
constexpr int kTreeRows = 128;        // rows of a tensor-core tile

__host__ __device__ __forceinline__ float* tree_part(const TreeArgs& a, int slot) {
  return a.part + (size_t)slot * a.slot_rows * a.c.head_dim;
}
__host__ __device__ __forceinline__ float* tree_part_stats(const TreeArgs& a, int slot) {
  return a.part + (size_t)2 * a.blocks * a.slot_rows * a.c.head_dim +
         (size_t)slot * a.slot_rows * 2;
}

// One sequence of a call.
struct TreeSeq {
  int s;        // its row in the cache
  int len;      // committed tokens
  int cnt;      // drafted tokens
  int lo;       // first tile (> 0 behind a window)
  int tiles;    // tiles of a unit; 0: nothing to do
  int row_tiles;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  TreeSeq r;
  r.s = cache_seq(a.c, a.seq, b);
  r.len = a.length[b];
  r.cnt = a.count ? a.count[b] : a.T;
  r.cnt = r.cnt < 0 ? 0 : r.cnt > a.T ? a.T : r.cnt;
  r.lo = 0;
  r.tiles = 0;
  r.row_tiles = (r.cnt + a.row_tokens - 1) / a.row_tokens;
  int err = r.s < 0 ? kCacheErrSeq : 0;
  if (!err && (r.len < 0 || (long long)r.len + r.cnt >
                                (long long)cache_held(a.c, r.s) * a.c.page_size))
    err = kCacheErrPage;
  if (err) {
    if (report) cache_error(a.c, err);
    return r;
  }
  if (r.cnt == 0) return r;
  if (a.window > 0 && r.len >= a.window) r.lo = (r.len - a.window + 1) / a.tile;
  r.tiles = (int)(((long long)r.len + r.cnt + a.tile - 1) / a.tile) - r.lo;
  return r;
}

__device__ __forceinline__ long long tree_work(const TreeArgs& a, const TreeSeq& r) {
  return (long long)r.tiles * r.row_tiles * a.c.kv_heads;
}

// Blocks that have a share, and the share of block c.
__device__ __forceinline__ long long tree_first(long long W, int G, int c) {
  return (W / G) * c + (W % G) * c / G;
}
// (W/G) c + floor((W % G) c / G) = floor(W c / G), without overflow.  The
// block of tile x: the largest c with floor(W c / G) <= x, found from the
// quotient and corrected by at most a step or two.
__device__ __forceinline__ int tree_block_of(long long W, int G, long long x) {
  int c = (int)((double)x * G / (double)W);
  if (c >= G) c = G - 1;
  while (c > 0 && tree_first(W, G, c) > x) --c;
  while (c + 1 < G && tree_first(W, G, c + 1) <= x) ++c;
  return c;
}

// A block's walk over its share, one unit at a time.
struct TreeWalk {
  long long pos, end;  // tiles of the line
  long long base;      // first tile of sequence b
  int b;
  TreeSeq q;
  // the current unit
  int h, rt;           // key head and row tile
  int first, n;        // its tiles here: first .. first + n - 1, counted from
                       // the unit's own first tile
  bool whole;          // all of the unit's tiles are here
  long long W;         // tiles of the line

  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (pos >= end) return false;
    long long work = tree_work(a, q);
    while (pos >= base + work) {
      base += work;
      if (++b >= a.B) return false;
      q = tree_seq(a, b, false);
      work = tree_work(a, q);
    }
    const long long at = pos - base;
    const int unit = (int)(at / q.tiles);
    first = (int)(at - (long long)unit * q.tiles);
    h = unit / q.row_tiles;
    rt = unit - h * q.row_tiles;
    const long long left = end - pos;
    n = q.tiles - first;
    if (n > left) n = (int)left;
    whole = n == q.tiles;
    pos += n;
    return true;
  }
};

// Every thread of the block calls this (blockDim.x a multiple of 32, all of
// `threads` of them): sums the work of the sequences and finds where this
// block's share starts.  `sums` is shared memory of 34 long longs.
__device__ __forceinline__ TreeWalk tree_start(const TreeArgs& a, long long* sums) {
  const int n = blockDim.x, t = threadIdx.x;
  const int per = (a.B + n - 1) / n;
  const int b0 = t * per, b1 = b0 + per < a.B ? b0 + per : a.B;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += tree_work(a, tree_seq(a, b, blockIdx.x == 0));
  const int lane = t & 31, warp = t >> 5;
  long long x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long before = 0, W = 0;
  for (int i = 0; i < n / 32; ++i) {
    if (i < warp) before += sums[i];
    W += sums[i];
  }
  before += x - mine;
  __syncthreads();
  const int G = W < a.blocks ? (int)W : a.blocks;
  TreeWalk w;
  w.pos = w.end = 0;
  w.base = 0;
  w.b = 0;
  w.h = w.rt = w.first = w.n = 0;
  w.whole = false;
  w.W = W;
  if ((int)blockIdx.x < G) {
    w.pos = tree_first(W, G, blockIdx.x);
    w.end = tree_first(W, G, blockIdx.x + 1);
    if (w.pos >= before && w.pos < before + mine) {
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const long long k = tree_work(a, tree_seq(a, b, false));
        if (w.pos < at + k) {
          sums[32] = b;
          sums[33] = at;
          break;
        }
        at += k;
      }
    }
  }
  __syncthreads();
  if ((int)blockIdx.x < G) {
    w.b = (int)sums[32];
    w.base = sums[33];
    w.q = tree_seq(a, w.b, false);
  }
  return w;
}

// One thread of every block, with a walk of its own that has not begun: what
// this block of the merge has to do.  The share's start cuts a unit when the
// first unit does not begin there; the unit is this block's to join when the
// share before it holds the unit's beginning.
__device__ __forceinline__ void tree_describe(const TreeArgs& a, TreeWalk w) {
  TreeJoin j{};
  const int c = blockIdx.x;
  const long long start = w.pos;
  if (w.next(a) && w.first > 0) {
    const int G = w.W < a.blocks ? (int)w.W : a.blocks;
    const long long us = start - w.first, before = tree_first(w.W, G, c - 1);
    if (before <= us) {
      j.b = w.b;
      j.h = w.h;
      j.t0 = w.rt * a.row_tokens;
      const int tokens = w.q.cnt - j.t0 < a.row_tokens ? w.q.cnt - j.t0 : a.row_tokens;
      j.rows = tokens * a.group;
      j.first = c - 1;
      j.slot = 2 * (c - 1) + (before == us ? 0 : 1);
      j.last = tree_block_of(w.W, G, us + w.q.tiles - 1);
    }
  }
  a.join[c] = j;
}

// The drafted tokens that token t of sequence b sees.
__device__ __forceinline__ uint64_t tree_mask(const TreeArgs& a, int b, int t, int cnt) {
  const uint64_t m = a.mask ? a.mask[(size_t)b * a.mask_stride + t]
                            : (t == 63 ? ~0ull : (2ull << t) - 1);
  return cnt >= 64 ? m : m & ((1ull << cnt) - 1);
}

// The first committed token that token t of sequence b sees.
__device__ __forceinline__ int tree_window_lo(const TreeArgs& a, int b, int t, int len) {
  if (a.window <= 0) return 0;
  long long pos = a.position ? a.position[(size_t)b * a.T + t] : (long long)len + t;
  if (pos < len) pos = len;
  const long long lo = pos - a.window + 1;
  return lo < 0 ? 0 : lo > len ? len : (int)lo;
}

bool tree_tc_supported(const TreeArgs& a);
cudaError_t launch_tree_tc(TreeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_tree_ffma(TreeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_tree_merge(const TreeArgs& a, cudaStream_t stream);

}  // namespace dspark
