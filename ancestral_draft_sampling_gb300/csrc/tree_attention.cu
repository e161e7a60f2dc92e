// tree_attention.cu -- attention of drafted tokens over the paged cache on
// the FFMA units (float32, and the shapes that the tensor-core kernel does
// not take), and the merge of partial results.
//
// One pass over a unit's keys with the running maximum m and sum l of each
// row: for a tile, s = scale q.k, m' = max(m, max s), p = exp(s - m'),
// l' = l e^(m - m') + sum p, o' = o e^(m - m') + p v.  All of it is float32.
// Eight warps hold four rows each, so a row's statistics stay in one warp and
// its weights p never leave it but for a small buffer of its own; keys and
// values of a tile are shared.  A tile is 64 keys by 32 rows.  Bound by the
// FFMA rate and by shared memory (6 loads of 16 bytes for 32 multiply-adds of
// the scores, 2 for 16 of the sums).
#include "dspark_common.cuh"
#include "host_util.cuh"
#include "sm100_ptx.cuh"
#include "tree_attention.cuh"

namespace dspark {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 32, kTile = 64;

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void put4(float* p, float4 x) {
  *reinterpret_cast<float4*>(p) = x;
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// ND: chunks of 128 dims that a lane's four cover (1: D <= 128, 2: D <= 256).
template <typename T, int ND>
__global__ void __launch_bounds__(kThreads, ND == 1 ? 2 : 1)
    tree_ffma_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(16) float smem[];
  __shared__ TreeShare share;
  const int D = a.c.head_dim, DP = D + 4;  // padded rows: lanes on different banks
  float* qs = smem;                        // [kRows][DP], scaled
  float* ks = qs + kRows * DP;             // [kTile][DP]
  float* vs = ks + kTile * DP;             // [kTile][D]
  float* ps = vs + kTile * D;              // [kWarps][kTile][4]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* q = static_cast<const T*>(a.q);
  const T* pool = static_cast<const T*>(a.c.pool);
  float* pw = ps + warp * kTile * 4;
  follow();
  tree_start(a, share);
  TreeWalk w = share.walk;
  if (threadIdx.x == kThreads - 1) tree_describe(a, w);
  bool is_first = true;
  for (bool some = w.n > 0; some; some = w.next(a)) {
    const int t0 = w.rt * a.row_tokens;
    const int rows = (w.q.cnt - t0 < a.row_tokens ? w.q.cnt - t0 : a.row_tokens) * a.group;
    const int head0 = w.h * a.group;
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
      float4 x = make_float4(0, 0, 0, 0);
      if (r < rows) {
        const int t = t0 + r / a.group, g = r % a.group;
        x = load4(q + (((size_t)w.b * a.T + t) * a.heads + head0 + g) * D + d);
        x = make_float4(x.x * a.scale, x.y * a.scale, x.z * a.scale, x.w * a.scale);
      }
      *reinterpret_cast<float4*>(qs + r * DP + d) = x;
    }
    // the warp's four rows
    float m[4], l[4];
    float4 o[4][ND];
    uint64_t bits[4];
    int lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = warp * 4 + i;
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int n = 0; n < ND; ++n) o[i][n] = make_float4(0, 0, 0, 0);
      bits[i] = 0;
      lo[i] = w.q.len;
      if (r < rows) {
        const int t = t0 + r / a.group;
        bits[i] = tree_mask(a, w.b, t, w.q.cnt);
        lo[i] = tree_window_lo(a, w.b, t, w.q.len);
      }
    }
    const int total = w.q.len + w.q.cnt;
    for (int tile = 0; tile < w.n; ++tile) {
      const int j0 = (w.q.lo + w.first + tile) * kTile;
      __syncthreads();  // the last tile's keys and values are used up
      for (int i = threadIdx.x; i < 2 * kTile * (D / 4); i += kThreads) {
        const bool val = i >= kTile * (D / 4);
        const int e = val ? i - kTile * (D / 4) : i;
        const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
        float4 x = make_float4(0, 0, 0, 0);
        if (j0 + r < total) {
          const int page = cache_page(a.c, w.q.s, (j0 + r) / a.c.page_size, a.c.max_pages);
          if (page >= 0)
            x = load4(pool + cache_row(a.c, 2 * a.layer + (val ? 1 : 0), page, w.h,
                                       (j0 + r) % a.c.page_size) / sizeof(T) + d);
          else
            cache_error(a.c, kCacheErrPage);
        }
        if (val) *reinterpret_cast<float4*>(vs + r * D + d) = x;
        else *reinterpret_cast<float4*>(ks + r * DP + d) = x;
      }
      __syncthreads();
      if (warp * 4 >= rows) continue;
      float s[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.0f;
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = load4(ks + lane * DP + d), k1 = load4(ks + (lane + 32) * DP + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = load4(qs + (warp * 4 + i) * DP + d);
          s[i][0] = dot4(x, k0, s[i][0]);
          s[i][1] = dot4(x, k1, s[i][1]);
        }
      }
      uint64_t seen[4];  // the tile's keys that the row sees
      uint64_t all = ~0ull;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bool see[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int j = j0 + lane + 32 * n;
          see[n] = j < w.q.len ? j >= lo[i]
                               : j < total && ((bits[i] >> (j - w.q.len)) & 1);
          if (!see[n]) s[i][n] = -INFINITY;
        }
        seen[i] = __ballot_sync(0xffffffffu, see[0]) |
                  (uint64_t)__ballot_sync(0xffffffffu, see[1]) << 32;
        all &= seen[i];
        float top = fmaxf(s[i][0], s[i][1]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float now = fmaxf(m[i], top);
        const float keep = m[i] == now ? 1.0f : expf(m[i] - now);
        const float p0 = see[0] && s[i][0] != -INFINITY ? expf(s[i][0] - now) : 0.0f;
        const float p1 = see[1] && s[i][1] != -INFINITY ? expf(s[i][1] - now) : 0.0f;
        float sum = p0 + p1;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[i] = l[i] * keep + sum;
        m[i] = now;
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          o[i][n].x *= keep;
          o[i][n].y *= keep;
          o[i][n].z *= keep;
          o[i][n].w *= keep;
        }
        pw[lane * 4 + i] = p0;
        pw[(lane + 32) * 4 + i] = p1;
      }
      __syncwarp();
      // a key that a row does not see is left out, whatever its values hold
#pragma unroll 4
      for (int j = 0; j < kTile; ++j) {
        const float4 p = load4(pw + j * 4);
        const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          const int d = n * 128 + lane * 4;
          if (d < D) {
            const float4 v = load4(vs + j * D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (all != ~0ull && !((seen[i] >> j) & 1)) continue;
              o[i][n].x = fmaf(pr[i], v.x, o[i][n].x);
              o[i][n].y = fmaf(pr[i], v.y, o[i][n].y);
              o[i][n].z = fmaf(pr[i], v.z, o[i][n].z);
              o[i][n].w = fmaf(pr[i], v.w, o[i][n].w);
            }
          }
        }
      }
      __syncwarp();
    }
    const int slot = 2 * blockIdx.x + (is_first ? 0 : 1);
    is_first = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = warp * 4 + i;
      if (r >= rows) break;
      const int t = t0 + r / a.group, g = r % a.group;
      const size_t row = ((size_t)w.b * a.T + t) * a.heads + head0 + g;
      const float inv = w.whole ? (l[i] == 0.0f ? 0.0f : 1.0f / l[i]) : 1.0f;
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        const int d = n * 128 + lane * 4;
        if (d >= D) continue;
        const float4 x = make_float4(o[i][n].x * inv, o[i][n].y * inv, o[i][n].z * inv,
                                     o[i][n].w * inv);
        if (w.whole) put4(static_cast<T*>(a.out) + row * D + d, x);
        else put4(tree_part(a, slot) + (size_t)r * D + d, x);
      }
      if (lane == 0) {
        if (!w.whole) {
          float* st = tree_part_stats(a, slot) + 2 * r;
          st[0] = m[i];
          st[1] = l[i];
        } else if (a.lse) {
          a.lse[row] = l[i] == 0.0f ? -INFINITY : m[i] + logf(l[i]);
        }
      }
    }
  }
}

// Joins the partial results of the units that several blocks worked on: a
// warp for each row, o = sum_c e^(m_c - M) o_c / sum_c e^(m_c - M) l_c over
// the unit's blocks c in order, M the largest m_c.
constexpr int kMergeWarps = 4, kMergeBatch = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  follow();
  const TreeJoin j = a.join[blockIdx.x + 1];  // nothing cuts the line's start
  const int lane = threadIdx.x & 31, D = a.c.head_dim;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (r >= j.rows) return;
  const int c0 = j.first, c1 = j.last, slot0 = j.slot;
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32)
    M = fmaxf(M, tree_part_stats(a, c == c0 ? slot0 : 2 * c)[2 * r]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float L = 0.0f;
  float4 o[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
  for (int cb = c0; cb <= c1; cb += 32) {
    const int n = c1 - cb + 1 < 32 ? c1 - cb + 1 : 32;
    float wt = 0.0f, lw = 0.0f;
    if (lane < n) {
      const int c = cb + lane;
      const float* st = tree_part_stats(a, c == c0 ? slot0 : 2 * c) + 2 * r;
      wt = st[0] == M ? 1.0f : exp2f((st[0] - M) * a.stat_log2);  // saw nothing: 0
      if (M == -INFINITY) wt = 0.0f;
      lw = wt * st[1];
    }
    for (int i0 = 0; i0 < n; i0 += kMergeBatch) {  // loads of a batch in flight
      float4 x[kMergeBatch][2];
#pragma unroll
      for (int i = 0; i < kMergeBatch; ++i) {
        const int c = cb + i0 + i;
        const float* part = tree_part(a, c == c0 ? slot0 : 2 * c) + (size_t)r * D;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int d = k * 128 + lane * 4;
          x[i][k] = make_float4(0, 0, 0, 0);
          if (i0 + i < n && d < D) x[i][k] = load4(part + d);
        }
      }
#pragma unroll
      for (int i = 0; i < kMergeBatch; ++i) {
        if (i0 + i >= n) break;
        const float wi = __shfl_sync(0xffffffffu, wt, i0 + i);
        L += __shfl_sync(0xffffffffu, lw, i0 + i);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          o[k].x = fmaf(wi, x[i][k].x, o[k].x);
          o[k].y = fmaf(wi, x[i][k].y, o[k].y);
          o[k].z = fmaf(wi, x[i][k].z, o[k].z);
          o[k].w = fmaf(wi, x[i][k].w, o[k].w);
        }
      }
    }
  }
  const size_t row =
      ((size_t)j.b * a.T + j.t0 + r / a.group) * a.heads + j.h * a.group + r % a.group;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = k * 128 + lane * 4;
    if (d < D)
      put4(static_cast<T*>(a.out) + row * D + d,
           make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
  }
  if (lane == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : M * a.stat_ln + logf(L);
}

// Dynamic shared memory a block may have beside its few static words.
constexpr int kMaxDynamic = 232448 - 1024;

template <typename T, int ND>
cudaError_t launch_ffma(const TreeArgs& a, size_t smem, cudaStream_t stream) {
  static std::once_flag once[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [] {
    cudaFuncSetAttribute(tree_ffma_kernel<T, ND>,
                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMaxDynamic);
  });
  return launch_behind(tree_ffma_kernel<T, ND>, a.blocks, kThreads, smem, stream, a);
}

}  // namespace

cudaError_t launch_tree_ffma(TreeArgs& a, int sms, cudaStream_t stream) {
  const int D = a.c.head_dim;
  a.tile_shift = 6;
  static_assert(kTile == 1 << 6, "tile");
  a.row_tokens = kRows / a.group;
  a.row_tiles = (a.T + a.row_tokens - 1) / a.row_tokens;
  a.slot_rows = (a.T < a.row_tokens ? a.T : a.row_tokens) * a.group;
  a.stat_log2 = 1.4426950408889634f;
  a.stat_ln = 1.0f;
  const size_t smem = sizeof(float) * ((size_t)(kRows + kTile) * (D + 4) +
                                       (size_t)kTile * D + kWarps * kTile * 4);
  // two blocks a multiprocessor where shared memory allows it (D <= 128)
  a.blocks = (smem * 2 + 4096 <= (size_t)kMaxDynamic ? 2 : 1) *
             (sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks);
  if (a.c.dtype == DSPARK_F32)
    return D <= 128 ? launch_ffma<float, 1>(a, smem, stream)
                    : launch_ffma<float, 2>(a, smem, stream);
  return D <= 128 ? launch_ffma<__nv_bfloat16, 1>(a, smem, stream)
                  : launch_ffma<__nv_bfloat16, 2>(a, smem, stream);
}

cudaError_t launch_tree_merge(const TreeArgs& a, cudaStream_t stream) {
  if (a.blocks < 2) return cudaSuccess;
  const dim3 grid(a.blocks - 1, (a.slot_rows + kMergeWarps - 1) / kMergeWarps);
  return launch_behind(a.c.dtype == DSPARK_F32 ? tree_merge_kernel<float>
                                               : tree_merge_kernel<__nv_bfloat16>,
                       grid, 32 * kMergeWarps, 0, stream, a);
}

}  // namespace dspark
