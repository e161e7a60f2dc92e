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
  int tile_shift;  // log2 of the keys of a tile
  int row_tokens;  // drafted tokens of a row tile
  int row_tiles;   // of T tokens
  int slot_rows;   // rows of a partial result
  struct TreeJoin* join;  // [G] what block c of the merge has to do
  // [2 G][slot_rows][D] sums, then [2 G][slot_rows][2]: maxima (in units of
  // log2) and sums of weights
  float* part;
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

// What is loaded for it, apart from what is made of that: a walk loads the
// next sequence's numbers while it is still at work on this one.
struct TreeRaw {
  int s, len, cnt, held;
};

__device__ __forceinline__ TreeRaw tree_load(const TreeArgs& a, int b) {
  TreeRaw r;
  r.s = cache_seq(a.c, a.seq, b);
  r.len = a.length[b];
  r.cnt = a.count ? a.count[b] : a.T;
  r.held = r.s < 0 ? 0 : a.c.page_count[r.s];
  return r;
}

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, const TreeRaw& w, bool report) {
  TreeSeq r;
  r.s = w.s;
  r.len = w.len;
  r.cnt = w.cnt < 0 ? 0 : w.cnt > a.T ? a.T : w.cnt;
  r.lo = 0;
  r.tiles = 0;
  r.row_tiles = 1;
  if (r.cnt > a.row_tokens) r.row_tiles = (uint32_t)(r.cnt + a.row_tokens - 1) / (uint32_t)a.row_tokens;
  const int held = w.held < 0 ? 0 : w.held > a.c.max_pages ? a.c.max_pages : w.held;
  int err = r.s < 0 ? kCacheErrSeq : 0;
  // a table row holds at most 2^30 tokens
  if (!err && (r.len < 0 || r.len > (1 << 30) || r.len + r.cnt > held * a.c.page_size))
    err = kCacheErrPage;
  if (err) {
    if (report) cache_error(a.c, err);
    return r;
  }
  if (r.cnt == 0) return r;
  if (a.window > 0 && r.len >= a.window) r.lo = (r.len - a.window + 1) >> a.tile_shift;
  r.tiles = ((r.len + r.cnt - 1) >> a.tile_shift) + 1 - r.lo;
  return r;
}

__device__ __forceinline__ long long tree_work(const TreeArgs& a, const TreeSeq& r) {
  return (long long)(r.row_tiles * a.c.kv_heads) * r.tiles;
}

// The line's tiles are counted in 32 bits (more than 2^31 of them, some ten
// seconds of work, are refused): code comes from memory while a block waits
// for it, and a 64-bit division is a hundred instructions.

// Where share c of W tiles over G blocks starts: floor(W c / G); c <= G <= 320.
__device__ __forceinline__ int tree_first(int W, int G, int c) {
  const uint32_t q = (uint32_t)W / (uint32_t)G, r = (uint32_t)W - q * G;
  return (int)(q * c + r * c / (uint32_t)G);
}

// A block's walk over its share, one unit at a time.
struct TreeWalk {
  int pos, end;        // tiles of the line
  int base;            // first tile of sequence b
  int W;               // tiles of the line
  int b;
  TreeSeq q;
  TreeRaw ahead;       // of sequence b + 1
  // the current unit
  int h, rt;           // key head and row tile
  int first, n;        // its tiles here: first .. first + n - 1, counted from
                       // the unit's own first tile
  bool whole;          // all of the unit's tiles are here

  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (pos >= end) return false;
    int work = q.row_tiles * a.c.kv_heads * q.tiles;
    while (pos >= base + work) {
      base += work;
      if (++b >= a.B) return false;
      q = tree_seq(a, ahead, false);
      if (b + 1 < a.B) ahead = tree_load(a, b + 1);
      work = q.row_tiles * a.c.kv_heads * q.tiles;
    }
    const uint32_t at = (uint32_t)(pos - base);
    const int unit = (int)(at / (uint32_t)q.tiles);
    first = (int)at - unit * q.tiles;
    h = unit;
    rt = 0;
    if (q.row_tiles > 1) {
      h = (int)((uint32_t)unit / (uint32_t)q.row_tiles);
      rt = unit - h * q.row_tiles;
    }
    const int left = end - pos;
    n = q.tiles - first;
    if (n > left) n = left;
    whole = n == q.tiles;
    pos += n;
    return true;
  }
};

// What the threads of a block tell each other when they find its share.
struct TreeShare {
  long long sums[32];
  TreeWalk walk;
};

// Every thread of the block calls this (blockDim.x a multiple of 32): sums the
// work of the sequences and finds where this block's share starts.  Leaves the
// walk in sh, on its first unit (n = 0: there is none), which one thread finds
// for all.  The block is synchronised twice.
__device__ __forceinline__ void tree_start(const TreeArgs& a, TreeShare& sh) {
  const int n = blockDim.x, t = threadIdx.x;
  const int per = a.B <= n ? 1 : (int)((uint32_t)(a.B + n - 1) / (uint32_t)n);
  const int b0 = t * per, b1 = b0 + per < a.B ? b0 + per : a.B;
  long long work = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b)
    work += tree_work(a, tree_seq(a, tree_load(a, b), blockIdx.x == 0));
  const int lane = t & 31, warp = t >> 5;
  long long x = work;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  if (lane == 31) sh.sums[warp] = x;
  __syncthreads();
  long long before = x - work, all = 0;
#pragma unroll 1
  for (int i = 0; i < n / 32; ++i) {
    const long long v = sh.sums[i];
    if (i < warp) before += v;
    all += v;
  }
  TreeWalk w{};
  if (all > 0x7fffffffLL) {
    if (blockIdx.x == 0 && t == 0) cache_error(a.c, kCacheErrPage);
    all = 0;
  }
  w.W = (int)all;
  const int G = w.W < a.blocks ? w.W : a.blocks;
  const bool some = (int)blockIdx.x < G;
  if (some) {
    w.pos = tree_first(w.W, G, blockIdx.x);
    w.end = tree_first(w.W, G, blockIdx.x + 1);
    if (w.pos >= before && w.pos < before + work) {  // one thread
      w.base = (int)before;
      w.b = b0;
      w.q = tree_seq(a, tree_load(a, b0), false);
      if (b0 + 1 < a.B) w.ahead = tree_load(a, b0 + 1);
      w.next(a);
      sh.walk = w;
    }
  } else if (t == 0) {
    sh.walk = w;
  }
  __syncthreads();
}

// One thread of every block, with the walk on its first unit: what this block
// of the merge has to do.  The share's start cuts a unit when the first unit
// does not begin there; the unit is this block's to join when the share before
// it holds the unit's beginning.
__device__ __forceinline__ void tree_describe(const TreeArgs& a, const TreeWalk& w) {
  TreeJoin j{};
  const int c = blockIdx.x;
  if (w.n > 0 && w.first > 0) {
    const int G = w.W < a.blocks ? w.W : a.blocks;
    const int us = w.pos - w.n - w.first, before = tree_first(w.W, G, c - 1);
    if (before <= us) {
      j.b = w.b;
      j.h = w.h;
      j.t0 = w.rt * a.row_tokens;
      const int tokens = w.q.cnt - j.t0 < a.row_tokens ? w.q.cnt - j.t0 : a.row_tokens;
      j.rows = tokens * a.group;
      j.first = c - 1;
      j.slot = 2 * (c - 1) + (before == us ? 0 : 1);
      j.last = c;
#pragma unroll 1
      while (j.last + 1 < G && tree_first(w.W, G, j.last + 1) < us + w.q.tiles) ++j.last;
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

bool tree_tc_supported(const TreeArgs& a);
cudaError_t launch_tree_tc(TreeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_tree_ffma(TreeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_tree_merge(const TreeArgs& a, cudaStream_t stream);

}  // namespace dspark
