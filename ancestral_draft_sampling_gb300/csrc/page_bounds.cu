// page_bounds.cu -- the smallest and largest keys of the pages that a call's
// tokens have filled, for each layer, key head and dimension: what the
// selection of pages scores them by.
//
// A minimum and a maximum of numbers of the cache's type is one of them, so
// nothing is rounded, and the order does not matter.  A NaN among the keys makes
// both NaN.
//
// Bound by HBM: every key of the filled pages is read once.  A warp takes one
// page of one head (page_size rows of head_dim, which lie together), with 16
// bytes a lane and eight rows in flight each; the (page, layer, head) units of
// all sequences form one line that the warps go through in strides, so one long
// prompt among short steps occupies the whole GPU.
#include <climits>

#include "cache.cuh"
#include "host_util.cuh"

namespace dspark {
namespace {

constexpr int kMaxB = DSPARK_CACHE_MAX_B;
constexpr int kThreads = 256, kAhead = 8;

// Four 32-bit words of keys: minima and maxima that a NaN wins.
template <typename T>
struct Range;
template <>
struct Range<float> {
  static constexpr uint32_t least = 0xff800000u, most = 0x7f800000u;  // -inf, inf
  static __device__ __forceinline__ uint32_t min(uint32_t x, uint32_t y) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
    return __float_as_uint(d);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t x, uint32_t y) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
    return __float_as_uint(d);
  }
};
template <>
struct Range<__nv_bfloat16> {
  static constexpr uint32_t least = 0xff80ff80u, most = 0x7f807f80u;
  static __device__ __forceinline__ uint32_t min(uint32_t x, uint32_t y) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
    return d;
  }
  static __device__ __forceinline__ uint32_t max(uint32_t x, uint32_t y) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
    return d;
  }
};

struct Rows {
  int seq[kMaxB];         // table rows
  int from[kMaxB];        // first filled page
  int offset[kMaxB + 1];  // filled pages of the rows before
  int warps[33];
};

// The pages that row b has filled: those that end in (start, length].
__device__ __forceinline__ int filled(const BoundsArgs& a, int b, Rows& sh, bool report) {
  const int s = cache_seq(a.c, a.seq, b), start = a.start[b], len = a.length[b];
  int err = s < 0 ? kCacheErrSeq : 0;
  // a table row holds at most 2^30 tokens
  if (!err && (start < 0 || len < 0 || len > (1 << 30) ||
               len > cache_held(a.c, s) * a.c.page_size))
    err = kCacheErrPage;
  sh.seq[b] = s;
  sh.from[b] = 0;
  if (err) {
    if (report) cache_error(a.c, err);
    return 0;
  }
  int slot;
  sh.from[b] = (int)page_of(a.c, (uint32_t)start, slot);
  const int n = (int)page_of(a.c, (uint32_t)len, slot) - sh.from[b];
  return n > 0 ? n : 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const __grid_constant__ BoundsArgs a) {
  using R = Range<T>;
  __shared__ Rows sh;
  follow();
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x; b < a.B; b += kThreads) sh.offset[b] = filled(a, b, sh, blockIdx.x == 0);
  __syncthreads();
  if ((long long)a.B * a.c.max_pages > INT_MAX) {  // the line is counted in 32 bits
    long long all = 0;
    for (int b = 0; b < a.B; ++b) all += sh.offset[b];
    if (all > INT_MAX) {
      if (blockIdx.x == 0 && threadIdx.x == 0) cache_error(a.c, kCacheErrPage);
      return;
    }
  }
  row_offsets(sh.offset, sh.offset, a.B, sh.warps);
  const uint32_t pages = sh.offset[a.B];
  const int words = a.c.head_dim * (int)sizeof(T) / 16;  // of a row
  const int rows = words < 32 ? 32 / words : 1;          // that a warp reads at a time
  const int row0 = words < 32 ? lane / words : 0, word0 = words < 32 ? lane - row0 * words : lane;
  // the warp's units: page, then layer and head
  const int each = a.c.layers * a.c.kv_heads;
  const int stride = gridDim.x * (kThreads / 32);
  const int page_step = stride / each, rest_step = stride - page_step * each;
  const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  uint32_t page = unit / each;
  int rest = unit - (int)page * each;
  const char* pool = static_cast<const char*>(a.c.pool);
  while (page < pages) {
    const int b = row_of(sh.offset, a.B, (int)page);
    const int id = cache_page(a.c, sh.seq[b], sh.from[b] + (int)page - sh.offset[b], a.c.max_pages);
    const int layer = rest / a.c.kv_heads, head = rest - layer * a.c.kv_heads;
    if (id < 0) {
      if (lane == 0) cache_error(a.c, kCacheErrPage);
    } else {
      const uint4* keys = reinterpret_cast<const uint4*>(pool + cache_row(a.c, 2 * layer, id, head, 0));
      uint4* out = reinterpret_cast<uint4*>(a.bounds + bounds_row(a.c, layer, id, head));
      for (int w0 = 0; w0 < words; w0 += 32) {  // one pass but for rows above 512 bytes
        const int w = w0 + word0;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = R::most;
          hi[i] = R::least;
        }
        if (row0 < rows && w < words) {
#pragma unroll 1
          for (int r = row0; r < a.c.page_size; r += kAhead * rows) {
            uint4 x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {  // a row read twice changes nothing
              const int at = r + k * rows;
              x[k] = keys[(size_t)(at < a.c.page_size ? at : r) * words + w];
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                lo[i] = R::min(lo[i], u[i]);
                hi[i] = R::max(hi[i], u[i]);
              }
            }
          }
        }
        // the rows that other lanes have read of the same word, to the first row's lanes
        const uint32_t lo0[4] = {lo[0], lo[1], lo[2], lo[3]}, hi0[4] = {hi[0], hi[1], hi[2], hi[3]};
#pragma unroll 1
        for (int k = 1; k < rows; ++k) {
          const int from = (lane + k * words) & 31;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = R::min(lo[i], __shfl_sync(0xffffffffu, lo0[i], from));
            hi[i] = R::max(hi[i], __shfl_sync(0xffffffffu, hi0[i], from));
          }
        }
        if (row0 == 0 && w < words) {
          out[w] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          out[words + w] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
      }
    }
    page += page_step;
    rest += rest_step;
    if (rest >= each) {
      rest -= each;
      ++page;
    }
  }
}

}  // namespace

cudaError_t launch_cache_bounds(const BoundsArgs& a, int sms, cudaStream_t stream) {
  const auto kernel = a.c.dtype == DSPARK_F32 ? bounds_kernel<float> : bounds_kernel<__nv_bfloat16>;
  return launch_behind(kernel, 4 * sms, kThreads, 0, stream, a);
}

}  // namespace dspark
