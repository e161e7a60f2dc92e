// part_attention.cu -- what stands before and behind the attention over part of
// the cache (tree_attention_tc.cuh, tree_attention_ffma.cuh).
//
// Selected pages: the lists of a sequence's tokens mostly name the same pages.
// They are made into one list for each key head, each page with a word that says
// which tokens see it, so that a page is read once for all its tokens' rows
// together (88 sequences with 8 tokens that choose 32 of 40 pages each: 4.4 GB
// less than token by token).  Order and repetition in the lists do not matter.
//
// Shared prefixes: softmax(q K^T) V over a sequence's keys is joined from that
// over its group's prefix and that over what follows, by the maxima m and sums l
// of both: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  The prefix is one
// item whose rows are those of all the group's sequences, so its keys are read
// once for 128 or 256 rows, and its products fill the tensor cores' tiles; prefixes
// and the rest are one line of tiles, which all blocks share.
#include "dspark_common.cuh"
#include "host_util.cuh"
#include "part_attention.cuh"

namespace dspark {
namespace {

constexpr int kMaxB = DSPARK_CACHE_MAX_B;
constexpr float kLn2 = 0.6931471805599453f;

// What a call says of a sequence; s < 0 or cnt < 0: it is not computed.
struct Held {
  int s, len, cnt, held;
};
__device__ __forceinline__ Held find_held(const TreeArgs& a, int b, bool report) {
  const TreeRaw w = tree_load(a, b);
  Held r{w.s, w.len, w.cnt < 0 ? 0 : w.cnt > a.T ? a.T : w.cnt, 0};
  r.held = w.held < 0 ? 0 : w.held > a.c.max_pages ? a.c.max_pages : w.held;
  int err = r.s < 0 ? kCacheErrSeq : 0;
  // a table row holds at most 2^30 tokens
  if (!err && (r.len < 0 || r.len > (1 << 30) || r.len + r.cnt > r.held * a.c.page_size))
    err = kCacheErrPage;
  if (err) {
    if (report) cache_error(a.c, err);
    r.cnt = -1;
  }
  return r;
}

__device__ __forceinline__ void put_item(const TreeArgs& a, int i, const TreeItem& x) {
  const int4* from = reinterpret_cast<const int4*>(&x);
  int4* to = reinterpret_cast<int4*>(const_cast<TreeItem*>(a.items) + i);
  to[0] = from[0];
  to[1] = from[1];
  to[2] = from[2];
  const_cast<long long*>(a.item_work)[i] =
      (long long)x.tiles * x.row_tiles * (x.h < 0 ? a.c.kv_heads : 1);
}

// ---------------------------------------------------------- selected pages
constexpr int kListThreads = 128, kRange = 1024;

__global__ void __launch_bounds__(kListThreads) sparse_items_kernel(const __grid_constant__ SparseArgs p) {
  __shared__ uint32_t seen[2][kRange];  // which tokens see a page of the range
  __shared__ int warps[33];
  const TreeArgs& a = p.a;
  follow();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int item = b * a.c.kv_heads + h;
  const Held q = find_held(a, b, h == 0 && tid == 0);
  TreeItem x{};
  x.list = (long long)item * p.room;
  x.b = b;
  x.h = h;
  if (q.cnt > 0) {
    int rest;
    const int F = (int)page_of(a.c, (uint32_t)q.len, rest);
    int32_t* list = const_cast<int32_t*>(a.page_list) + x.list;
    uint64_t* bits = const_cast<uint64_t*>(a.page_bits) + x.list;
    const int lists = p.lists == 1 ? 1 : q.cnt, entries = lists * p.count;
    const size_t step = (size_t)a.c.kv_heads * p.count;  // between the lists of two tokens
    const int32_t* from = p.pages + ((size_t)b * p.lists * a.c.kv_heads + h) * p.count;
    int n = 0;
    for (int r0 = 0; r0 < F; r0 += kRange) {
      for (int i = tid; i < 2 * kRange; i += kListThreads) (&seen[0][0])[i] = 0;
      __syncthreads();
      bool any = false;
      for (int e = tid; e < entries; e += kListThreads) {
        const int t = (int)((uint32_t)e / (uint32_t)p.count);
        const int page = from[t * step + (e - t * p.count)];
        if (page >= F && r0 == 0) cache_error(a.c, kCacheErrPage);
        if (page < r0 || page >= F || page >= r0 + kRange) continue;
        any = true;
        if (p.lists == 1) {
          seen[0][page - r0] = seen[1][page - r0] = ~0u;
        } else {
          atomicOr(&seen[t >> 5][page - r0], 1u << (t & 31));
        }
      }
      if (!__syncthreads_or(any)) continue;
      constexpr int kEach = kRange / kListThreads;
      int mine = 0;
      for (int i = 0; i < kEach; ++i) {
        const int at = tid * kEach + i;
        mine += (seen[0][at] | seen[1][at]) != 0;
      }
      int total;
      int at = n + block_exclusive(mine, warps, total);
      for (int i = 0; i < kEach; ++i) {
        const int k = tid * kEach + i;
        const uint64_t m = (uint64_t)seen[1][k] << 32 | seen[0][k];
        if (m) {
          list[at] = cache_page(a.c, q.s, r0 + k, q.held);  // -1 is reported where it is read
          bits[at] = m;
          ++at;
        }
      }
      n += total;
      __syncthreads();
    }
    // behind them the partly filled page and the drafted tokens
    const int last = (q.len + q.cnt - 1) / a.c.page_size;
    for (int i = F + tid; i <= last; i += kListThreads) list[n + i - F] = cache_page(a.c, q.s, i, q.held);
    x.hide = n * a.c.page_size;
    x.len = x.hide + rest;
    x.cnt = q.cnt;
    x.tokens = q.cnt;
    x.tiles = ((x.len + x.cnt - 1) >> a.tile_shift) + 1;
    x.row_tiles = (q.cnt + a.row_tokens - 1) / a.row_tokens;
  }
  if (tid == 0) put_item(a, item, x);
}

// ---------------------------------------------------------- shared prefixes
constexpr int kItemThreads = 1024;

__global__ void __launch_bounds__(kItemThreads) prefix_items_kernel(const __grid_constant__ PrefixArgs p) {
  __shared__ int len[kMaxB];     // committed tokens; -1: nothing to do
  __shared__ int shared[kMaxB];  // of these, those of the group's prefix
  __shared__ int group[kMaxB];
  const TreeArgs& a = p.a;
  follow();
  const int tid = threadIdx.x;  // kMaxB sequences at most
  Held q{-1, 0, -1, 0};
  if (tid < a.B) {
    q = find_held(a, tid, true);
    len[tid] = q.cnt > 0 ? q.len : -1;
    shared[tid] = 0;
    group[tid] = -1;
  }
  int from = 0, to = 0, n = 0;
  bool fine = true;
  if (tid < p.groups) {
    from = p.group_start[tid];
    to = p.group_start[tid + 1];
    n = p.prefix[tid];
    fine = 0 <= from && from <= to && to <= a.B && n >= 0;
  }
  fine = __syncthreads_and(fine);
  if (!fine && tid == 0) cache_error(a.c, kCacheErrGroup);
  if (tid < p.groups) {
    TreeItem x{};
    x.b = from;
    x.h = -1;
    x.kind = kTreeShared;
    if (fine && to - from > 1 && n > 0) {
      const int s = cache_seq(a.c, a.seq, from);
      if (s < 0 || n > (1 << 30) || n > cache_held(a.c, s) * a.c.page_size) {
        cache_error(a.c, kCacheErrGroup);
      } else {
        int users = 0;
        for (int b = from; b < to; ++b) {
          if (len[b] < 0) continue;
          if (len[b] < n) {
            cache_error(a.c, kCacheErrGroup);
            continue;
          }
          shared[b] = n;
          group[b] = tid;
          ++users;
        }
        if (users > 0) {
          x.list = (long long)s * a.c.max_pages;
          x.len = n;
          x.tokens = (to - from) * a.T;
          x.tiles = ((n - 1) >> a.tile_shift) + 1;
          x.row_tiles = (x.tokens + a.row_tokens - 1) / a.row_tokens;
        }
      }
    }
    put_item(a, tid, x);
  }
  __syncthreads();
  if (tid < a.B) {
    TreeItem x{};
    x.b = tid;
    x.h = -1;
    x.kind = kTreeOwn;
    if (q.cnt > 0) {
      x.list = (long long)q.s * a.c.max_pages;
      x.hide = shared[tid];
      x.lo = x.hide >> a.tile_shift;
      x.len = q.len;
      x.cnt = q.cnt;
      x.tokens = q.cnt;
      x.tiles = ((q.len + q.cnt - 1) >> a.tile_shift) + 1 - x.lo;
      x.row_tiles = (q.cnt + a.row_tokens - 1) / a.row_tokens;
    }
    put_item(a, p.groups + tid, x);
    p.group_of[tid] = group[tid];
  }
}

// A row's parts of one item: of blocks first .. first + n - 1 of the attention,
// or, if n = 1, the whole.
struct Parts {
  int n, first, slot, r;  // slot: of the first block's part; r: the row there
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

constexpr int kJoinWarps = 4, kBatch = 4;

template <typename T, int ND>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_kernel(const __grid_constant__ PrefixArgs p) {
  const TreeArgs& a = p.a;
  follow();
  const size_t row = (size_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= tree_rows(a)) return;
  const int lane = threadIdx.x & 31, D = a.c.head_dim;
  const uint32_t bt = (uint32_t)(row / (uint32_t)a.heads), head = (uint32_t)(row - (size_t)bt * a.heads);
  const int b = (int)(bt / (uint32_t)a.T), t = (int)(bt - (uint32_t)b * a.T);
  const int h = (int)(head / (uint32_t)a.group), gh = (int)head - h * a.group;
  using Source = TreeSource<true>;
  const TreeItem own = Source::load(a, p.groups + b);
  const long long all = a.item_base[a.item_count];
  if (own.tiles == 0 || t >= own.tokens || all > 0x7fffffffLL) return;
  const int W = (int)all, G = W < a.blocks ? W : a.blocks;
  auto block_of = [&](int at) { return (int)((((long long)at + 1) * G - 1) / W); };
  auto parts_of = [&](const TreeItem& x, int item, int token) {
    Parts r;
    const int rt = token / a.row_tokens;
    const int us = (int)a.item_base[item] + (h * x.row_tiles + rt) * x.tiles;
    r.first = block_of(us);
    r.n = block_of(us + x.tiles - 1) - r.first + 1;
    r.slot = 2 * r.first + (tree_first(W, G, r.first) == us ? 0 : 1);
    r.r = (token - rt * a.row_tokens) * a.group + gh;
    return r;
  };
  const Parts mine = parts_of(own, p.groups + b, t);
  Parts theirs{0, 0, 0, 0};
  const int g = p.group_of[b];
  if (g >= 0) {
    const TreeItem x = Source::load(a, g);
    theirs = parts_of(x, g, (b - x.b) * a.T + t);
  }
  const int parts = mine.n + theirs.n;
  auto sums = [&](int i) -> const float* {
    const Parts& k = i < mine.n ? mine : theirs;
    if (k.n == 1) return tree_whole(a, i < mine.n ? kTreeOwn : kTreeShared, row);
    const int j = i < mine.n ? i : i - mine.n;
    return tree_part(a, j == 0 ? k.slot : 2 * (k.first + j)) + (size_t)k.r * D;
  };
  auto stats = [&](int i) {
    if (i >= parts) return make_float2(-INFINITY, 0.0f);
    const Parts& k = i < mine.n ? mine : theirs;
    const int j = i < mine.n ? i : i - mine.n;
    const float* at = k.n == 1 ? tree_whole_stats(a, i < mine.n ? kTreeOwn : kTreeShared, row)
                               : tree_part_stats(a, j == 0 ? k.slot : 2 * (k.first + j)) + 2 * k.r;
    return *reinterpret_cast<const float2*>(at);
  };
  float M = -INFINITY, L = 0.0f;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, stats(i).x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float4 o[ND];
#pragma unroll
  for (int k = 0; k < ND; ++k) o[k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int p0 = 0; p0 < parts; p0 += kBatch) {
    float4 x[kBatch][ND];
    float2 st[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      st[i] = stats(p0 + i);
      const float* at = p0 + i < parts ? sums(p0 + i) : nullptr;
#pragma unroll
      for (int k = 0; k < ND; ++k) {
        const int d = k * 128 + lane * 4;
        x[i][k] = make_float4(0, 0, 0, 0);
        if (at && d < D) x[i][k] = load4(at + d);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // a part that saw nothing weighs nothing
      const float w = M == -INFINITY ? 0.0f : st[i].x == M ? 1.0f : exp2f(st[i].x - M);
      L += w * st[i].y;
#pragma unroll
      for (int k = 0; k < ND; ++k) {
        o[k].x = fmaf(w, x[i][k].x, o[k].x);
        o[k].y = fmaf(w, x[i][k].y, o[k].y);
        o[k].z = fmaf(w, x[i][k].z, o[k].z);
        o[k].w = fmaf(w, x[i][k].w, o[k].w);
      }
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
  for (int k = 0; k < ND; ++k) {
    const int d = k * 128 + lane * 4;
    if (d < D)
      put4(static_cast<T*>(a.out) + row * D + d,
           make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
  }
  if (lane == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
}

}  // namespace

cudaError_t launch_sparse_items(const SparseArgs& a, cudaStream_t stream) {
  return launch_behind(sparse_items_kernel, dim3(a.a.c.kv_heads, a.a.B), kListThreads, 0, stream, a);
}

cudaError_t launch_prefix_items(const PrefixArgs& a, cudaStream_t stream) {
  return launch_behind(prefix_items_kernel, 1, kItemThreads, 0, stream, a);
}

cudaError_t launch_prefix_join(const PrefixArgs& a, cudaStream_t stream) {
  const size_t rows = (size_t)a.a.B * a.a.T * a.a.heads;
  const unsigned blocks = (unsigned)((rows + kJoinWarps - 1) / kJoinWarps);
  const bool wide = a.a.c.head_dim > 128;
  const auto kernel = a.a.c.dtype == DSPARK_F32
                          ? (wide ? prefix_join_kernel<float, 2> : prefix_join_kernel<float, 1>)
                          : (wide ? prefix_join_kernel<__nv_bfloat16, 2> : prefix_join_kernel<__nv_bfloat16, 1>);
  return launch_behind(kernel, blocks, 32 * kJoinWarps, 0, stream, a);
}

}  // namespace dspark
