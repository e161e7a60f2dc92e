// part_attention.cu -- what stands before and behind the attention over part of
// the cache (tree_attention_tc.cuh, tree_attention_ffma.cuh).
//
// Selected pages: the lists of a sequence's tokens mostly name the same pages.
// They are made into one list for each key head, each page with a word that says
// which tokens see it, so that a page is read once for all its tokens' rows
// together (88 sequences with one to 8 tokens that choose 32 of 40 pages each: 0.9 GB,
// and 3.3 token by token).  Order and repetition in the lists do not matter.
//
// Shared prefixes: softmax(q K^T) V over a sequence's keys is joined from that
// over its group's prefix and that over what follows, by the maxima m and sums l
// of both: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  The prefix is one
// item whose rows are those of all the group's sequences, so its keys are read
// once for 128 or 256 rows, and its products fill the tensor cores' tiles.  Prefixes
// and the rest are one line of tiles, which all blocks share, or, where they want
// different forms of the kernel, a line and a launch each (PrefixArgs::two).
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
  const long long work =
      x.tiles == 0 ? 0 : (long long)(x.tiles + a.extra) * x.row_tiles * (x.h < 0 ? a.c.kv_heads : 1);
  const_cast<long long*>(a.item_work)[i] = work;
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
    // one list in ascending order, as it is selected, needs no sorting out
    bool sorted = lists == 1;
    if (sorted) {
      for (int i = tid; i < p.count && sorted; i += kListThreads) {
        const int page = from[i], before = i > 0 ? from[i - 1] : -1;
        sorted = page < F && (page < 0 || i == 0 || (before >= 0 && before < page));
        n += page >= 0;
      }
      sorted = __syncthreads_and(sorted);
    }
    if (sorted) {
      int total;
      block_exclusive(n, warps, total);
      n = total;
      for (int i = tid; i < n; i += kListThreads) {
        list[i] = cache_page(a.c, q.s, from[i], q.held);  // -1 is reported where it is read
        bits[i] = ~0ull;
      }
    } else {
      n = 0;
      for (int r0 = 0; r0 < F || r0 == 0; r0 += kRange) {  // without full pages too: entries are looked at
        const int each = ((F - r0 < kRange ? F - r0 : kRange) + kListThreads - 1) / kListThreads;
        for (int i = tid; i < each * kListThreads; i += kListThreads) seen[0][i] = seen[1][i] = 0;
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
        int mine = 0;
        for (int i = 0; i < each; ++i) mine += (seen[0][tid * each + i] | seen[1][tid * each + i]) != 0;
        int total;
        int at = n + block_exclusive(mine, warps, total);
        for (int i = 0; i < each; ++i) {
          const int k = tid * each + i;
          const uint64_t m = (uint64_t)seen[1][k] << 32 | seen[0][k];
          if (m) {
            list[at] = cache_page(a.c, q.s, r0 + k, q.held);
            bits[at] = m;
            ++at;
          }
        }
        n += total;
        __syncthreads();
      }
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
  __shared__ int start[kMaxB + 1];  // of the groups
  __shared__ int prefix[kMaxB];     // their shared tokens; 0: each sequence by itself
  __shared__ int used[kMaxB];       // by a sequence
  const TreeArgs &a = p.shared, &own = p.two ? p.own : p.shared;
  follow();
  const int tid = threadIdx.x;  // kMaxB sequences at most
  Held q{-1, 0, -1, 0};
  if (tid < a.B) q = find_held(a, tid, true);
  bool fine = true;
  if (tid < p.groups) {
    const int from = p.group_start[tid], to = p.group_start[tid + 1], n = p.prefix[tid];
    fine = 0 <= from && from <= to && to <= a.B && n >= 0;
    start[tid] = from;
    if (tid + 1 == p.groups) start[p.groups] = to;
    prefix[tid] = to > from ? n : 0;
    used[tid] = 0;
  }
  fine = __syncthreads_and(fine);
  if (!fine && tid == 0) cache_error(a.c, kCacheErrGroup);
  long long list = 0;
  if (fine && tid < p.groups && prefix[tid] > 0 && start[tid + 1] - start[tid] > 1) {
    const int s = cache_seq(a.c, a.seq, start[tid]), n = prefix[tid];
    list = (long long)s * a.c.max_pages;
    if (s < 0 || n > a.length[start[tid]] || n > (1 << 30) || n > cache_held(a.c, s) * a.c.page_size) {
      cache_error(a.c, kCacheErrGroup);
      prefix[tid] = 0;
    }
  }
  __syncthreads();
  int g = -1, hide = 0;
  if (fine && q.cnt > 0 && tid >= start[0] && tid < start[p.groups]) {
    g = row_of(start, p.groups, tid);
    hide = prefix[g];
    const bool less = q.len < hide;
    if (less) cache_error(a.c, kCacheErrGroup);
    if (less || start[g + 1] - start[g] == 1) hide = 0;  // a row alone has nobody to share with
    if (hide > 0) used[g] = 1;
  }
  __syncthreads();
  if (tid < p.groups) {
    TreeItem x{};
    x.b = start[tid];
    x.h = -1;
    x.kind = kTreeShared;
    if (used[tid]) {
      x.list = list;
      x.len = prefix[tid];
      x.tokens = (start[tid + 1] - start[tid]) * a.T;
      x.tiles = ((x.len - 1) >> a.tile_shift) + 1;
      x.row_tiles = (x.tokens + a.row_tokens - 1) / a.row_tokens;
    }
    put_item(a, tid, x);
  }
  if (tid < a.B) {
    TreeItem x{};
    x.b = tid;
    x.h = -1;
    x.kind = kTreeOwn;
    if (q.cnt > 0) {
      x.list = (long long)q.s * a.c.max_pages;
      x.hide = hide;
      x.lo = x.hide >> own.tile_shift;
      x.len = q.len;
      x.cnt = q.cnt;
      x.tokens = q.cnt;
      x.tiles = ((q.len + q.cnt - 1) >> own.tile_shift) + 1 - x.lo;
      x.row_tiles = (q.cnt + own.row_tokens - 1) / own.row_tokens;
    }
    put_item(own, p.two ? tid : p.groups + tid, x);
    p.group_of[tid] = hide > 0 ? g : -1;
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

// A row's parts: some of what its sequence has of its own, then some of the prefix.
// A warp takes four rows, with a lane for each row of 8 parts, which finds that part and
// its statistics, and the loads of four parts of all in flight.  Bound by latency:
// what a line's blocks have of it is found without a division, which the attention's
// first block has made (88 single tokens of 64 heads in nine parts: 11 us, 13.4 with six
// divisions a lane and half as many loads in flight; 16384 rows in two or three parts:
// 15, and 18 with two rows a warp and eight parts).
constexpr int kJoinWarps = 4, kJoinRows = 4, kJoinParts = 32 / kJoinRows, kJoinBatch = 4;

template <typename T, int ND>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_kernel(const __grid_constant__ PrefixArgs p) {
  const TreeArgs &a = p.shared, &line = p.two ? p.own : p.shared;
  follow();
  const int lane = threadIdx.x & 31, D = a.c.head_dim, sub = lane / kJoinRows;
  const int h = blockIdx.y, b = blockIdx.z, r0 = (blockIdx.x * kJoinWarps + (threadIdx.x >> 5)) * kJoinRows;
  using Source = TreeSource<true>;
  const int own_item = p.two ? b : p.groups + b, g = p.group_of[b];
  const TreeItem own = Source::load(line, own_item);
  const long long own_all = line.item_base[line.item_count], all = a.item_base[a.item_count];
  const long long own_each = line.item_base[line.item_count + 1], each = a.item_base[a.item_count + 1];
  const int own_base = (int)line.item_base[own_item], rows = own.tokens * a.group;
  const TreeItem shared = Source::load(a, g < 0 ? 0 : g);
  const int base = (int)a.item_base[g < 0 ? 0 : g];
  if (own.tiles == 0 || r0 >= rows || own_all > 0x7fffffffLL || all > 0x7fffffffLL) return;
  // this lane's row of the warp's (the last one again behind it)
  const int mine = r0 + lane % kJoinRows < rows ? r0 + lane % kJoinRows : rows - 1;
  const int t = (int)((uint32_t)mine / (uint32_t)a.group), gh = mine - t * a.group;
  const size_t row = ((size_t)b * a.T + t) * a.heads + h * a.group + gh;
  auto parts_of = [&](const TreeArgs& l, int W, long long shares, const TreeItem& x, int from, int token) {
    Parts r;
    const int G = W < l.blocks ? W : l.blocks, q = (int)shares, rest = (int)(shares >> 32);
    const float part = __fdividef(1.0f, (float)G), per = __fdividef((float)G, (float)W);
    // tree_first: rest c < 2^15, so half a unit outweighs float's rounding
    static_assert(kTreeMaxBlocks * kTreeMaxBlocks < 1 << 15, "rest and c are below the blocks");
    auto first_of = [&](int c) { return q * c + (int)(((float)(rest * c) + 0.5f) * part); };
    // the block of a place, found from beside it
    auto block_of = [&](int at) {
      int c = (int)((float)at * per);
      c = c >= G ? G - 1 : c;
      while (c > 0 && first_of(c) > at) --c;
      while (c + 1 < G && first_of(c + 1) <= at) ++c;
      return c;
    };
    // tokens of a group are fewer than 2^17
    const int rt = (int)(((float)token + 0.5f) * __fdividef(1.0f, (float)l.row_tokens));
    const int us = from + (h * x.row_tiles + rt) * (x.tiles + l.extra);
    r.first = block_of(us + l.extra);
    r.n = block_of(us + l.extra + x.tiles - 1) - r.first + 1;
    r.slot = 2 * r.first + (first_of(r.first) >= us ? 0 : 1);
    r.r = (token - rt * l.row_tokens) * l.group + gh;
    return r;
  };
  const Parts x = parts_of(line, (int)own_all, own_each, own, own_base, t);
  Parts y{0, 0, 0, 0};
  if (g >= 0) y = parts_of(a, (int)all, each, shared, base, (b - shared.b) * a.T + t);
  const int parts = x.n + y.n;
  const int most = __reduce_max_sync(0xffffffffu, parts);
  float M = -INFINITY, L = 0.0f;
  float4 o[kJoinRows][ND];
#pragma unroll
  for (int n = 0; n < kJoinRows; ++n)
#pragma unroll
    for (int k = 0; k < ND; ++k) o[n][k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int p0 = 0; p0 < most; p0 += kJoinParts) {
    // part p0 + sub of the lane's row
    unsigned long long sums = 0;
    float2 st = make_float2(-INFINITY, 0.0f);
    const int i = p0 + sub;
    if (i < parts) {
      const bool second = i >= x.n;
      const int n = second ? y.n : x.n, first = second ? y.first : x.first, r = second ? y.r : x.r;
      const int j = second ? i - x.n : i, kind = second ? kTreeShared : kTreeOwn;
      const TreeArgs& l = second ? a : line;
      const int slot = j == 0 ? (second ? y.slot : x.slot) : 2 * (first + j);
      const float* stats = n == 1 ? tree_whole_stats(a, kind, row) : tree_part_stats(l, slot) + 2 * r;
      sums = reinterpret_cast<unsigned long long>(n == 1 ? tree_whole(a, kind, row) : tree_part(l, slot) + (size_t)r * D);
      st = *reinterpret_cast<const float2*>(stats);
    }
    const int here = most - p0 < kJoinParts ? most - p0 : kJoinParts;
    float w = 0.0f;
#pragma unroll 1
    for (int q0 = 0; q0 < here; q0 += kJoinBatch) {
      float4 v[kJoinBatch][kJoinRows][ND];
#pragma unroll
      for (int q = 0; q < kJoinBatch; ++q)
#pragma unroll
        for (int n = 0; n < kJoinRows; ++n) {
          const float* from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, sums, (q0 + q) * kJoinRows + n));
#pragma unroll
          for (int k = 0; k < ND; ++k) {
            v[q][n][k] = make_float4(0, 0, 0, 0);
            if (from && k * 128 + lane * 4 < D) v[q][n][k] = load4(from + k * 128 + lane * 4);
          }
        }
      if (q0 == 0) {  // while they are under way: the weights of these parts
        float now = st.x;
#pragma unroll
        for (int k = kJoinRows; k < 32; k <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, k));
        now = fmaxf(now, M);
        // a part that saw nothing weighs nothing
        w = now == -INFINITY ? 0.0f : st.x == now ? 1.0f : exp2f(st.x - now);
        const float keep = M == now ? 1.0f : exp2f(M - now);
        float sum = w * st.y;
#pragma unroll
        for (int k = kJoinRows; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        L = L * keep + sum;
        M = now;
        if (p0 > 0) {
#pragma unroll
          for (int n = 0; n < kJoinRows; ++n) {
            const float f = __shfl_sync(0xffffffffu, keep, n);
#pragma unroll
            for (int k = 0; k < ND; ++k) o[n][k] = make_float4(o[n][k].x * f, o[n][k].y * f, o[n][k].z * f, o[n][k].w * f);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kJoinBatch; ++q)
#pragma unroll
        for (int n = 0; n < kJoinRows; ++n) {
          const float f = __shfl_sync(0xffffffffu, w, (q0 + q) * kJoinRows + n);
#pragma unroll
          for (int k = 0; k < ND; ++k) {
            o[n][k].x = fmaf(f, v[q][n][k].x, o[n][k].x);
            o[n][k].y = fmaf(f, v[q][n][k].y, o[n][k].y);
            o[n][k].z = fmaf(f, v[q][n][k].z, o[n][k].z);
            o[n][k].w = fmaf(f, v[q][n][k].w, o[n][k].w);
          }
        }
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  if (lane < kJoinRows && r0 + lane < rows && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
#pragma unroll
  for (int n = 0; n < kJoinRows; ++n) {
    const float f = __shfl_sync(0xffffffffu, inv, n);
    const size_t to = __shfl_sync(0xffffffffu, (unsigned long long)row, n);
    if (r0 + n >= rows) break;
#pragma unroll
    for (int k = 0; k < ND; ++k) {
      const int d = k * 128 + lane * 4;
      if (d < D)
        put4(static_cast<T*>(a.out) + to * D + d,
             make_float4(o[n][k].x * f, o[n][k].y * f, o[n][k].z * f, o[n][k].w * f));
    }
  }
}

}  // namespace

cudaError_t launch_sparse_items(const SparseArgs& a, cudaStream_t stream) {
  return launch_behind(sparse_items_kernel, dim3(a.a.c.kv_heads, a.a.B), kListThreads, 0, stream, a);
}

cudaError_t launch_prefix_items(const PrefixArgs& a, cudaStream_t stream) {
  return launch_behind(prefix_items_kernel, 1, kItemThreads, 0, stream, a);
}

cudaError_t launch_prefix_join(const PrefixArgs& a, cudaStream_t stream) {
  const TreeArgs& l = a.shared;
  constexpr int rows = kJoinRows * kJoinWarps;
  const dim3 blocks((l.T * l.group + rows - 1) / rows, l.c.kv_heads, l.B);
  const bool wide = l.c.head_dim > 128;
  const auto kernel = l.c.dtype == DSPARK_F32
                          ? (wide ? prefix_join_kernel<float, 2> : prefix_join_kernel<float, 1>)
                          : (wide ? prefix_join_kernel<__nv_bfloat16, 2> : prefix_join_kernel<__nv_bfloat16, 1>);
  return launch_behind(kernel, blocks, 32 * kJoinWarps, 0, stream, a);
}

}  // namespace dspark
