// cache.cuh -- the paged key/value cache as the kernels see it: addresses of
// a sequence's tokens, the device error word, and block-wide scans.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/dspark.h"
#include "sm100_ptx.cuh"

namespace dspark {

// Words of `control`: the device error word, the number of free pages, the
// ticket of a call's last block, and scratch behind them that a call writes
// before it reads it.
constexpr int kCtlError = 0, kCtlFree = 1, kCtlTicket = 2;
constexpr int kCtlScratch = 64;  // 2 * DSPARK_CACHE_MAX_B words

enum CacheError : int {
  kCacheErrSeq = 6,
  kCacheErrPage = 7,
  kCacheErrFull = 8,
  kCacheErrPath = 9,
  kCacheErrPosition = 10,
  kCacheErrFork = 11,
};

__device__ __forceinline__ void cache_error(const dspark_cache& c, int code) {
  c.control[kCtlError] = code;
}

__host__ __device__ __forceinline__ int dtype_bytes(dspark_dtype t) {
  return t == DSPARK_F32 ? 4 : 2;
}

// The sequence of row b of a call, or -1.
__device__ __forceinline__ int cache_seq(const dspark_cache& c,
                                         const int32_t* seq, int b) {
  const int s = seq ? seq[b] : b;
  return s >= 0 && s < c.max_seqs ? s : -1;
}

// Pages that sequence s holds, within the table row whatever the array says.
__device__ __forceinline__ int cache_held(const dspark_cache& c, int s) {
  const int n = c.page_count[s];
  return n < 0 ? 0 : n > c.max_pages ? c.max_pages : n;
}

// Page i of sequence s, or -1 if it holds none there.
__device__ __forceinline__ int cache_page(const dspark_cache& c, int s, int i,
                                          int held) {
  if (i < 0 || i >= held) return -1;
  const int p = c.block_table[(size_t)s * c.max_pages + i];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// The page of token x of a sequence, and its place there.  Page sizes are
// mostly powers of two, and a division is 25 instructions: in kernels this
// short they come from memory, one cache line after another.
__device__ __forceinline__ uint32_t page_of(const dspark_cache& c, uint32_t x, int& slot) {
  const uint32_t n = (uint32_t)c.page_size;
  if ((n & (n - 1)) == 0) {
    slot = (int)(x & (n - 1));
    return x >> (31 - __clz(n));
  }
  const uint32_t p = x / n;
  slot = (int)(x - p * n);
  return p;
}
// Pages that hold x tokens.
__device__ __forceinline__ uint32_t pages_for(const dspark_cache& c, uint32_t x) {
  int slot;
  return x == 0 ? 0u : page_of(c, x - 1, slot) + 1;
}

// Bytes from the start of the pool to a token of one head: plane 2 layer
// (keys) or 2 layer + 1 (values).
__host__ __device__ __forceinline__ size_t cache_row(const dspark_cache& c,
                                                     int plane, int page,
                                                     int head, int slot) {
  return ((((size_t)plane * c.num_pages + page) * c.kv_heads + head) *
              c.page_size + slot) * ((size_t)c.head_dim * dtype_bytes(c.dtype));
}

// Every kernel of the cache starts with this: the next one may be set up from
// now on, and the ones before have finished and their writes are visible.
__device__ __forceinline__ void follow() {
  sm100::launch_dependents();
  sm100::grid_dependency_wait();
}

// Two float32 operations in one instruction, on a pair in 64 bits.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Exclusive sum over the block's threads (a multiple of 32, at most 1024);
// `total` is the block's sum.  `warps` is shared memory of 33 ints; the call
// synchronises the block before and after using it.
__device__ __forceinline__ int block_exclusive(int v, int* warps, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int n = blockDim.x >> 5;
    int w = lane < n ? warps[lane] : 0;
    int y = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += o;
    }
    if (lane < n) warps[lane] = y - w;
    if (lane == 31) warps[32] = y;
  }
  __syncthreads();
  total = warps[32];
  return warps[warp] + x - v;
}

cudaError_t launch_cache_init(const dspark_cache& c, cudaStream_t stream);
cudaError_t launch_cache_reserve(const dspark_cache& c, const int32_t* seq,
                                 const int32_t* length, int tokens, int B,
                                 cudaStream_t stream);
cudaError_t launch_cache_release(const dspark_cache& c, const int32_t* seq,
                                 int B, cudaStream_t stream);
cudaError_t launch_cache_fork(const dspark_cache& c, const int32_t* parent,
                              const int32_t* child, const int32_t* length,
                              int B, cudaStream_t stream);
cudaError_t launch_cache_accept(const dspark_cache& c, const int32_t* seq,
                                const int32_t* length, const int32_t* accepted,
                                const int32_t* path, int path_width, int extra,
                                int tokens, int B, int32_t* new_length,
                                cudaStream_t stream);

struct AppendArgs {
  dspark_cache c;
  int layer;
  const int32_t *seq, *length, *count;
  const char *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const float *q_weight, *k_weight;
  float eps;
  const float* cos_sin;
  int max_position, rot, interleaved;
  const int32_t* position;
  int B, T, heads;
  char* q_out;
};
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream);

}  // namespace dspark
