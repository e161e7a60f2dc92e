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

// What part of the cache a unit's rows attend to where that is not a sequence's
// whole one: an item, made by a kernel before the attention.  Its keys are those
// of a list of pages, in the list's order; of them the first `hide` are not seen
// (kind kTreeOwn) or ruled page by page (TreeArgs::page_bits), the others to `len`
// are seen, and behind these lie `cnt` drafted ones, ruled by the mask.
struct TreeItem {
  long long list;  // its first page in TreeArgs::page_list
  int lo;          // first tile
  int hide;        // see above
  int len, cnt;
  int tokens;      // of rows: the first is token 0 of sequence b
  int tiles, row_tiles;
  int b;
  int h;           // its key head; -1: all
  int kind;
};
static_assert(sizeof(TreeItem) == 48, "three 16-byte loads");
constexpr int kTreeSparse = 0;  // selected pages: results like those of a sequence
constexpr int kTreeShared = 1;  // a prefix that sequences share, and
constexpr int kTreeOwn = 2;     // what a sequence has behind it: partial results

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
  int most;        // drafted tokens of a sequence or item, at most
  struct TreeJoin* join;  // [G] what block c of the merge has to do
  // [2 G][slot_rows][D] sums, then [2 G][slot_rows][2]: maxima (in units of
  // log2) and sums of weights
  float* part;
  // items (the kernels' other form)
  const TreeItem* items;
  const long long* item_work;  // tiles of each
  int item_count;
  const int32_t* page_list;
  const uint64_t* page_bits;   // beside page_list: bit t: token t sees the page
  // out, or null: [item_count + 2] the line's place where an item starts, all places,
  // and floor(places / blocks) with the rest of that division above it
  long long* item_base;
  // kinds kTreeShared and kTreeOwn: results of units that one block has whole,
  // by row [B][T][heads] and kind: sums [2][rows][D], maxima and sums [2][rows][2]
  float* whole;
  // The end of a unit and the start of the next cost as much as some tiles: each
  // unit of an item has so many places on the line before its own.
  int extra;
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

__device__ __forceinline__ size_t tree_rows(const TreeArgs& a) {
  return (size_t)a.B * a.T * a.heads;
}
__device__ __forceinline__ float* tree_whole(const TreeArgs& a, int kind, size_t row) {
  return a.whole + ((kind - 1) * tree_rows(a) + row) * a.c.head_dim;
}
__device__ __forceinline__ float* tree_whole_stats(const TreeArgs& a, int kind, size_t row) {
  return a.whole + 2 * tree_rows(a) * a.c.head_dim + ((kind - 1) * tree_rows(a) + row) * 2;
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

// Where a walk's units come from: the sequences of a call, or items.
template <bool kItems>
struct TreeSource {
  using Raw = TreeRaw;
  using Seq = TreeSeq;
  static __device__ __forceinline__ int count(const TreeArgs& a) { return a.B; }
  static __device__ __forceinline__ Raw load(const TreeArgs& a, int b) { return tree_load(a, b); }
  static __device__ __forceinline__ Seq make(const TreeArgs& a, const Raw& r) { return tree_seq(a, r, false); }
  static __device__ __forceinline__ long long work(const TreeArgs& a, int b) {
    return tree_work(a, tree_seq(a, tree_load(a, b), blockIdx.x == 0));
  }
  static __device__ __forceinline__ int work(const TreeArgs& a, const Seq& q) {
    return q.row_tiles * a.c.kv_heads * q.tiles;
  }
  static __device__ __forceinline__ int extra(const TreeArgs&) { return 0; }
  static __device__ __forceinline__ int head(const Seq&) { return 0; }
  static __device__ __forceinline__ int tokens(const Seq& q) { return q.cnt; }
  static __device__ __forceinline__ int row(const Seq&, int b) { return b; }
};
template <>
struct TreeSource<true> {
  using Raw = TreeItem;
  using Seq = TreeItem;
  static __device__ __forceinline__ int count(const TreeArgs& a) { return a.item_count; }
  static __device__ __forceinline__ Raw load(const TreeArgs& a, int b) {
    Raw r;
    const int4* p = reinterpret_cast<const int4*>(a.items + b);
    reinterpret_cast<int4*>(&r)[0] = p[0];
    reinterpret_cast<int4*>(&r)[1] = p[1];
    reinterpret_cast<int4*>(&r)[2] = p[2];
    return r;
  }
  static __device__ __forceinline__ Seq make(const TreeArgs&, const Raw& r) { return r; }
  static __device__ __forceinline__ long long work(const TreeArgs& a, int b) { return a.item_work[b]; }
  static __device__ __forceinline__ int work(const TreeArgs& a, const Seq& q) {
    return q.tiles == 0 ? 0 : q.row_tiles * (q.tiles + a.extra) * (q.h < 0 ? a.c.kv_heads : 1);
  }
  static __device__ __forceinline__ int extra(const TreeArgs& a) { return a.extra; }
  static __device__ __forceinline__ int head(const Seq& q) { return q.h < 0 ? 0 : q.h; }
  static __device__ __forceinline__ int tokens(const Seq& q) { return q.tokens; }
  static __device__ __forceinline__ int row(const Seq& q, int) { return q.b; }
};

// The line's tiles are counted in 32 bits (more than 2^31 of them, some ten
// seconds of work, are refused): code comes from memory while a block waits
// for it, and a 64-bit division is a hundred instructions.

// Where share c of W tiles over G blocks starts: floor(W c / G); c <= G <= kTreeMaxBlocks.
__device__ __forceinline__ int tree_first(int W, int G, int c) {
  const uint32_t q = (uint32_t)W / (uint32_t)G, r = (uint32_t)W - q * G;
  return (int)(q * c + r * c / (uint32_t)G);
}

// A block's walk over its share, one unit at a time.
template <bool kItems>
struct TreeWalk {
  using Source = TreeSource<kItems>;
  int pos, end;        // tiles of the line
  int base;            // first tile of sequence b
  int W;               // tiles of the line
  int b;
  typename Source::Seq q;
  typename Source::Raw ahead;       // of sequence b + 1
  // the current unit
  int h, rt;           // key head and row tile
  int first, n;        // its tiles here: first .. first + n - 1, counted from
                       // the unit's own first tile
  bool whole;          // all of the unit's tiles are here

  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if constexpr (kItems) {  // a share may end in the places before a unit's tiles
      do {
        if (!step(a)) {
          n = 0;
          return false;
        }
      } while (n == 0);
      return true;
    } else {
      return step(a);
    }
  }
  __device__ __forceinline__ bool step(const TreeArgs& a) {
    if (pos >= end) return false;
    int work = Source::work(a, q);
    while (pos >= base + work) {
      base += work;
      if (++b >= Source::count(a)) return false;
      q = Source::make(a, ahead);
      if (b + 1 < Source::count(a)) ahead = Source::load(a, b + 1);
      work = Source::work(a, q);
    }
    const uint32_t at = (uint32_t)(pos - base);
    const int extra = Source::extra(a), places = q.tiles + extra;
    const int unit = (int)(at / (uint32_t)places);
    first = (int)at - unit * places;
    h = unit;
    rt = 0;
    if (q.row_tiles > 1) {
      h = (int)((uint32_t)unit / (uint32_t)q.row_tiles);
      rt = unit - h * q.row_tiles;
    }
    h += Source::head(q);
    const int left = end - pos;
    n = places - first;
    if (n > left) n = left;
    pos += n;
    if constexpr (kItems) {
      const int last = first + n - extra;  // tiles before the share's end
      first = first > extra ? first - extra : 0;
      n = last > first ? last - first : 0;
    }
    whole = n == q.tiles;
    return true;
  }
};

// What the threads of a block tell each other when they find its share.
template <bool kItems>
struct TreeShare {
  long long sums[16];  // of the block's warps
  TreeWalk<kItems> walk;
};

// Every thread of the block calls this (blockDim.x a multiple of 32): sums the
// work of the sequences and finds where this block's share starts.  Leaves the
// walk in sh, on its first unit (n = 0: there is none), which one thread finds
// for all.  The block is synchronised twice.
template <bool kItems>
__device__ __forceinline__ void tree_start(const TreeArgs& a, TreeShare<kItems>& sh) {
  using Source = TreeSource<kItems>;
  const int n = blockDim.x, t = threadIdx.x, B = Source::count(a);
  const int per = B <= n ? 1 : (int)((uint32_t)(B + n - 1) / (uint32_t)n);
  const int b0 = t * per, b1 = b0 + per < B ? b0 + per : B;
  long long work = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b)
    work += Source::work(a, b);
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
  if (kItems && a.item_base && blockIdx.x == 0) {
    long long at = before;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      a.item_base[b] = at;
      at += Source::work(a, b);
    }
    if (t == 0) {
      a.item_base[B] = all;
      const uint32_t W = (uint32_t)all, G = W < (uint32_t)a.blocks ? (W ? W : 1u) : (uint32_t)a.blocks;
      a.item_base[B + 1] = (long long)(W / G) | (long long)(W - W / G * G) << 32;
    }
  }
  TreeWalk<kItems> w{};
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
      w.q = Source::make(a, Source::load(a, b0));
      if (b0 + 1 < B) w.ahead = Source::load(a, b0 + 1);
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
template <bool kItems>
__device__ __forceinline__ void tree_describe(const TreeArgs& a, const TreeWalk<kItems>& w) {
  using Source = TreeSource<kItems>;
  TreeJoin j{};
  const int c = blockIdx.x;
  if (w.n > 0 && w.first > 0) {
    const int G = w.W < a.blocks ? w.W : a.blocks, extra = Source::extra(a);
    const int us = w.pos - w.n - w.first - extra, before = tree_first(w.W, G, c - 1);
    if (before <= us + extra) {
      j.b = Source::row(w.q, w.b);
      j.h = w.h;
      j.t0 = w.rt * a.row_tokens;
      const int left = Source::tokens(w.q) - j.t0;
      const int tokens = left < a.row_tokens ? left : a.row_tokens;
      j.rows = tokens * a.group;
      j.first = c - 1;
      j.slot = 2 * (c - 1) + (before >= us ? 0 : 1);
      j.last = c;
#pragma unroll 1
      while (j.last + 1 < G && tree_first(w.W, G, j.last + 1) < us + extra + w.q.tiles) ++j.last;
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

// Whether the tensor-core kernel takes a cache.
bool tree_tc_supported(const TreeArgs& a);
// Whether its units of up to `tokens` tokens are narrow (tree_attention_tc.cuh).
bool tree_tc_narrow(const TreeArgs& a, int tokens);
// How the work is cut up, for units of up to `tokens` tokens.
void tree_tc_plan(TreeArgs& a, int tokens, int sms);
void tree_ffma_plan(TreeArgs& a, int tokens, int sms);
cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_ffma(const TreeArgs& a, cudaStream_t stream);
// The same over items, which may have heads of other sizes too.
bool items_tc_supported(const TreeArgs& a);
cudaError_t launch_items_tc(const TreeArgs& a, cudaStream_t stream);
cudaError_t launch_items_ffma(const TreeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_merge(const TreeArgs& a, cudaStream_t stream);

}  // namespace dspark
