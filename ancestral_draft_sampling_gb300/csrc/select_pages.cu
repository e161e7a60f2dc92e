// select_pages.cu -- the pages of a long context that a query's attention is
// to read: those whose bounds allow the largest products with it.
//
// A page's keys lie between lo and hi in each dimension, so no product of q with
// one of them exceeds s = sum_d max(q_d lo_d, q_d hi_d) = q+ . hi + q- . lo with
// q+ = max(q, 0) and q- = min(q, 0).  A list takes, for the query heads of one key
// head (of one token, or of all of a sequence's), the `count` pages with the
// largest max s.
//
// Which pages these are does not depend on the order of the sums: scores are
// made in float32, and where some lie so near the border between taken and not
// taken that their error could decide, those few are scored again in 64 bits
// (products of the inputs are exact there, sums to 2^-53).  The error of a score
// is below eps = D 2^-22 A, A = the largest sum of |q_d| times the largest |bound|:
// a product of the tensor cores adds 16 exact terms to a float32 sum, off by at
// most 17 truncations of 2^-24 A, and a score takes D / 8 of them, 2.1 D 2^-24 A
// together; the FFMA form makes D roundings.
//
// The scores are a pass over the bounds (2 D values a page and head against
// 2 D page_size of keys and values), bound by HBM for few query rows.  bfloat16
// with head_dim a multiple of 32 is multiplied by mma.sync straight from global
// memory: a row of 32 bounds is four lanes' 16 bytes, and since the order of a sum's
// terms is free, a lane's eight values serve as its parts of two operands.  (q+, q-
// and the bounds are bfloat16 numbers: nothing is rounded but the sums.)  Tiles in
// shared memory and tcgen05 would buy nothing: a page's 512 bytes a head are used by
// at most a few hundred rows.
#include <climits>
#include <cmath>

#include "dspark_common.cuh"
#include "host_util.cuh"
#include "select_pages.cuh"

namespace dspark {
namespace {

// One sequence: its table row and its full pages; F < 0: there is an error.
struct Seq {
  int s, F, tokens;
};
__device__ __forceinline__ Seq find_seq(const SelectArgs& a, int b, bool report) {
  Seq r;
  r.s = cache_seq(a.c, a.seq, b);
  const int len = a.length[b], n = a.tokens ? a.tokens[b] : a.T;
  r.tokens = n < 0 ? 0 : n > a.T ? a.T : n;
  r.F = -1;
  const int err = r.s < 0 ? kCacheErrSeq
                  : len < 0 || len > (1 << 30) || len > cache_held(a.c, r.s) * a.c.page_size
                      ? kCacheErrPage : 0;
  if (err) {
    if (report) cache_error(a.c, err);
    return r;
  }
  int slot;
  r.F = (int)page_of(a.c, (uint32_t)len, slot);
  return r;
}

__device__ __forceinline__ size_t list_row(const SelectArgs& a, int b, int t, int h) {
  return ((size_t)b * a.lists + t) * a.c.kv_heads + h;
}

// ------------------------------------------------------------------ scores
// A block takes a sequence's key head and a stretch of its pages, one after the
// other if the table is long; a warp scores 16 pages (8 on the FFMA units) at a time.
constexpr int kScoreThreads = 128, kScoreWarps = kScoreThreads / 32;

// A score as it is kept: what is not a number counts as the highest.
__device__ __forceinline__ float kept(float s) { return s == s ? s : INFINITY; }

__device__ __forceinline__ uint32_t max_nan2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
  return d;
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// The sums of |q|: tokens blockIdx.x, + gridDim.x .. of the block's key head, a
// warp for each.
template <typename T>
__device__ __forceinline__ void sum_queries(const SelectArgs& a, int b, int h, int tokens) {
  const int lane = threadIdx.x & 31, D = a.c.head_dim;
#pragma unroll 1
  for (int t = blockIdx.x + gridDim.x * (threadIdx.x >> 5); t < tokens; t += gridDim.x * kScoreWarps) {
    const size_t token = (size_t)b * a.T + t;
    const T* q = reinterpret_cast<const T*>(a.q) + (token * a.heads + (size_t)h * a.group) * D;
    float best = 0.0f;
#pragma unroll 4
    for (int g = 0; g < a.group; ++g) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = 4 * lane + 128 * k;
        if (d < D) {
          const float4 v = load4<T>(q + (size_t)g * D + d);
          x += fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w);
        }
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
      best = max_nan(best, x);
    }
    if (lane == 0) a.reach_q[token * a.c.kv_heads + h] = best;
  }
}

// c += a b: a 16 rows of 16, b 16 x 8, bfloat16, sums in float32.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 query rows that are worked on together; KD: head_dim / 32, or 0:
// any.
template <int NT, int KD>
__global__ void __launch_bounds__(kScoreThreads)
    score_mma_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kRows = 8 * NT, kPitch = kRows + 1;
  __shared__ float slab[kScoreWarps][16 * kPitch];
  follow();
  const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const Seq seq = find_seq(a, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (seq.F <= 0 || seq.tokens == 0) return;
  float* const mine = slab[warp];
  const int D = KD ? 32 * KD : a.c.head_dim, fit = kRows / a.group;  // tokens of a row tile
  const bool together = a.lists == 1;
  sum_queries<__nv_bfloat16>(a, b, h, seq.tokens);
#pragma unroll 1
  for (int page0 = (blockIdx.x * kScoreWarps + warp) * 16; page0 < seq.F; page0 += gridDim.x * kScoreWarps * 16) {
    const int j = lane & 15, pages = seq.F - page0;
    const int id = j < pages ? cache_page(a.c, seq.s, page0 + j, a.c.max_pages) : -1;
    if (j < pages && id < 0) cache_error(a.c, kCacheErrPage);
    const int id0 = __shfl_sync(0xffffffffu, id, gid), id1 = __shfl_sync(0xffffffffu, id, gid + 8);
    const uint4* k0 = reinterpret_cast<const uint4*>(a.bounds + bounds_row(a.c, a.layer, id0 < 0 ? 0 : id0, h)) + tig;
    const uint4* k1 = reinterpret_cast<const uint4*>(a.bounds + bounds_row(a.c, a.layer, id1 < 0 ? 0 : id1, h)) + tig;
    uint32_t top0 = 0, top1 = 0;  // the largest |bound| of both pages
    float run = -INFINITY;
#pragma unroll 1
    for (int t0 = 0; t0 < seq.tokens; t0 += fit) {
      const int tokens = seq.tokens - t0 < fit ? seq.tokens - t0 : fit;
      const uint4 none = make_uint4(0, 0, 0, 0);
      const uint4* q[NT];  // row 8 n + gid of the tile
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + gid, t = r / a.group;
        const size_t row = ((size_t)b * a.T + t0 + t) * a.heads + (size_t)h * a.group + (r - t * a.group);
        q[n] = t < tokens ? reinterpret_cast<const uint4*>(a.q + row * D * 2) + tig : nullptr;
      }
      float c[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll 4
      for (int k = 0; k < D / 32; ++k) {
        uint4 l0 = none, l1 = none, h0 = none, h1 = none;
        if (id0 >= 0) {
          l0 = k0[4 * k];
          h0 = k0[D / 8 + 4 * k];
        }
        if (id1 >= 0) {
          l1 = k1[4 * k];
          h1 = k1[D / 8 + 4 * k];
        }
        if (t0 == 0) {
          const uint32_t m = 0x7fff7fffu;
          const uint32_t x[8] = {l0.x, l0.y, l0.z, l0.w, h0.x, h0.y, h0.z, h0.w};
          const uint32_t y[8] = {l1.x, l1.y, l1.z, l1.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            top0 = max_nan2(top0, x[i] & m);
            top1 = max_nan2(top1, y[i] & m);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 x = q[n] ? q[n][4 * k] : none;
          mma16816(c[n], l0.x, l1.x, l0.y, l1.y, min_nan2(x.x, 0), min_nan2(x.y, 0));
          mma16816(c[n], l0.z, l1.z, l0.w, l1.w, min_nan2(x.z, 0), min_nan2(x.w, 0));
          mma16816(c[n], h0.x, h1.x, h0.y, h1.y, max_nan2(x.x, 0), max_nan2(x.y, 0));
          mma16816(c[n], h0.z, h1.z, h0.w, h1.w, max_nan2(x.z, 0), max_nan2(x.w, 0));
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine[(gid + (i >> 1) * 8) * kPitch + 8 * n + 2 * tig + (i & 1)] = c[n][i];
      __syncwarp();
      // the largest of a token's heads: a page a lane, every other token
      for (int t = lane >> 4; t < tokens; t += 2) {
        float best = -INFINITY;
        for (int g = 0; g < a.group; ++g) best = fmaxf(best, kept(mine[j * kPitch + t * a.group + g]));
        if (id < 0) best = -INFINITY;
        if (together) run = fmaxf(run, best);
        else if (j < pages) a.scores[list_row(a, b, t0 + t, h) * a.stride + page0 + j] = best;
      }
      __syncwarp();
    }
    if (together) {
      run = fmaxf(run, __shfl_xor_sync(0xffffffffu, run, 16));
      if (lane < 16 && j < pages) a.scores[list_row(a, b, 0, h) * a.stride + page0 + j] = run;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      top0 = max_nan2(top0, __shfl_xor_sync(0xffffffffu, top0, x));
      top1 = max_nan2(top1, __shfl_xor_sync(0xffffffffu, top1, x));
    }
    if (lane < 2) {
      const uint32_t x = lane ? top1 : top0;
      a.reach_k[((size_t)b * a.c.kv_heads + h) * a.reaches + page0 / kReachPages + lane] =
          max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
  }
}

// s + max(q lo, q hi) for finite numbers; where the bounds or q are not, every
// page is scored in 64 bits.
__device__ __forceinline__ float reach(float q, float lo, float hi, float s) {
  return fmaf(q, q < 0.0f ? lo : hi, s);
}

// The same on the FFMA units: four lanes share a page, and take eight query rows
// at a time.
template <typename T>
__global__ void __launch_bounds__(kScoreThreads)
    score_ffma_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kTake = 8, kPages = 8;
  static_assert(kPages == kReachPages, "a warp's pages");
  follow();
  const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3, D = a.c.head_dim;
  const Seq seq = find_seq(a, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (seq.F <= 0 || seq.tokens == 0) return;
  const bool together = a.lists == 1;
  sum_queries<T>(a, b, h, seq.tokens);
  const int rows = seq.tokens * a.group;
  const T* q = reinterpret_cast<const T*>(a.q) + ((size_t)b * a.T * a.heads + (size_t)h * a.group) * D;
#pragma unroll 1
  for (int page0 = (blockIdx.x * kScoreWarps + warp) * kPages; page0 < seq.F;
       page0 += gridDim.x * kScoreWarps * kPages) {
    const int j = page0 + gid;
    const int id = j < seq.F ? cache_page(a.c, seq.s, j, a.c.max_pages) : -1;
    if (j < seq.F && id < 0) cache_error(a.c, kCacheErrPage);
    const T* lo = reinterpret_cast<const T*>(a.bounds + bounds_row(a.c, a.layer, id < 0 ? 0 : id, h));
    float top = 0.0f, best = -INFINITY;
    int g = 0, t = 0;  // of the row that is next
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kTake) {
      float s[kTake];
      const T* at[kTake];
      int ta = t, ga = g;
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        s[i] = 0.0f;
        at[i] = q + ((size_t)ta * a.heads + ga) * D;
        if (r0 + i + 1 < rows && ++ga == a.group) {
          ga = 0;
          ++ta;
        }
      }
#pragma unroll 4
      for (int d = 4 * tig; d < D; d += 16) {
        const float4 l = load4<T>(lo + d), u = load4<T>(lo + D + d);
        if (r0 == 0 && id >= 0) {
          top = max_nan(top, max_nan(max_nan(fabsf(l.x), fabsf(l.y)), max_nan(fabsf(l.z), fabsf(l.w))));
          top = max_nan(top, max_nan(max_nan(fabsf(u.x), fabsf(u.y)), max_nan(fabsf(u.z), fabsf(u.w))));
        }
#pragma unroll
        for (int i = 0; i < kTake; ++i) {
          const float4 x = load4<T>(at[i] + d);
          s[i] = reach(x.x, l.x, u.x, s[i]);
          s[i] = reach(x.y, l.y, u.y, s[i]);
          s[i] = reach(x.z, l.z, u.z, s[i]);
          s[i] = reach(x.w, l.w, u.w, s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        s[i] += __shfl_xor_sync(0xffffffffu, s[i], 1);
        s[i] += __shfl_xor_sync(0xffffffffu, s[i], 2);
      }
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        if (r0 + i >= rows) break;
        best = fmaxf(best, kept(s[i]));
        if (++g == a.group) {
          if (!together) {
            if (tig == 0 && j < seq.F) a.scores[list_row(a, b, t, h) * a.stride + j] = id < 0 ? -INFINITY : best;
            best = -INFINITY;
          }
          g = 0;
          ++t;
        }
      }
    }
    if (together && tig == 0 && j < seq.F)
      a.scores[list_row(a, b, 0, h) * a.stride + j] = id < 0 ? -INFINITY : best;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (lane == 0) a.reach_k[((size_t)b * a.c.kv_heads + h) * a.reaches + page0 / kPages] = top;
  }
}

// --------------------------------------------------------------- selection
constexpr int kPickThreads = 256;
constexpr int kNear = 32;  // pages near the border that one warp ranks

__device__ __forceinline__ uint64_t ordered_bits64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return u >> 63 ? ~u : u | (1ull << 63);
}

// W warps that work on one list.
template <int W>
struct Team {
  struct Shared {
    uint32_t part[2][W];
    int n, near[kNear];
    uint64_t exact[kNear];
  };
  Shared& sh;
  int thread, turn = 0;
  __device__ __forceinline__ Team(Shared& s, int t) : sh(s), thread(t) {}
  __device__ __forceinline__ void sync() const {
    if (W > 1) __syncthreads();
    else __syncwarp();
  }
  template <typename F>
  __device__ __forceinline__ uint32_t join(uint32_t x, F f) {
    if (W == 1) return x;
    if ((thread & 31) == 0) sh.part[turn][thread >> 5] = x;
    __syncthreads();
    uint32_t y = sh.part[turn][0];
#pragma unroll
    for (int i = 1; i < W; ++i) y = f(y, sh.part[turn][i]);
    turn ^= 1;
    return y;
  }
  __device__ __forceinline__ uint32_t sum(uint32_t x) {
    return join(__reduce_add_sync(0xffffffffu, x), [](uint32_t p, uint32_t q) { return p + q; });
  }
  __device__ __forceinline__ uint32_t least(uint32_t x) {
    return join(__reduce_min_sync(0xffffffffu, x), [](uint32_t p, uint32_t q) { return p < q ? p : q; });
  }
  __device__ __forceinline__ uint32_t most(uint32_t x) {
    return join(__reduce_max_sync(0xffffffffu, x), [](uint32_t p, uint32_t q) { return p > q ? p : q; });
  }
};

// q times the bound that makes the larger product, exact.
__device__ __forceinline__ double larger(float q, float lo, float hi) {
  return (double)q * (q < 0.0f ? lo : hi);
}
// The same as whole multiples of 1 / scale (a power of two): the products of
// bfloat16 numbers are exact in float32, and those of float32 numbers with the
// remainder, which a fused product gives.
template <typename T>
__device__ __forceinline__ long long larger_fixed(float q, float lo, float hi, float scale) {
  const float x = q < 0.0f ? lo : hi, p = q * x;
  long long n = __float2ll_rn(p * scale);
  if (sizeof(T) == 4) n += __float2ll_rn(fmaf(q, x, -p) * scale);
  return n;
}

// The score of one page in 64 bits, by a whole warp: as a whole number of 1 / scale,
// whose sums are exact, or where scale is 0 (infinities, extreme sizes) in double.
// The 64-bit floating-point units have a thirty-second of the integer units' rate
// and bounded the selection: 5632 lists of 250 pages 67 -> 20 us.
template <typename T>
__device__ __noinline__ uint64_t exact_score(const SelectArgs& a, int b, int t0, int tokens, int h,
                                             int page, float scale, int lane) {
  const int D = a.c.head_dim;
  const T* lo = reinterpret_cast<const T*>(a.bounds + bounds_row(a.c, a.layer, page < 0 ? 0 : page, h));
  long long most = LLONG_MIN;
  double best = -INFINITY;
#pragma unroll 1
  for (int t = t0; t < t0 + tokens; ++t) {
    const T* q = reinterpret_cast<const T*>(a.q) +
                 (((size_t)b * a.T + t) * a.heads + (size_t)h * a.group) * D;
    if (scale > 0.0f) {
#pragma unroll 4
      for (int g = 0; g < a.group; ++g) {
        long long s = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int d = 4 * lane + 128 * k;
          if (d < D) {
            const float4 x = load4<T>(q + (size_t)g * D + d), l = load4<T>(lo + d), u = load4<T>(lo + D + d);
            s += larger_fixed<T>(x.x, l.x, u.x, scale) + larger_fixed<T>(x.y, l.y, u.y, scale) +
                 larger_fixed<T>(x.z, l.z, u.z, scale) + larger_fixed<T>(x.w, l.w, u.w, scale);
          }
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        most = s > most ? s : most;
      }
    } else {
#pragma unroll 1
      for (int g = 0; g < a.group; ++g) {
        double s = 0.0;
        for (int d = 4 * lane; d < D; d += 128) {
          const float4 x = load4<T>(q + (size_t)g * D + d), l = load4<T>(lo + d), u = load4<T>(lo + D + d);
          s += larger(x.x, l.x, u.x);
          s += larger(x.y, l.y, u.y);
          s += larger(x.z, l.z, u.z);
          s += larger(x.w, l.w, u.w);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        best = s == s ? fmax(best, s) : INFINITY;
      }
    }
  }
  // as bits whose order is that of the scores
  if (page < 0) return 0;
  return scale > 0.0f ? (uint64_t)most ^ (1ull << 63) : ordered_bits64(best);
}

// W warps a list, R scores a thread in registers (the rest is read from memory
// each time).
template <typename T, int W, int R>
__global__ void __launch_bounds__(kPickThreads) pick_pages_kernel(const __grid_constant__ SelectArgs a) {
  using TeamW = Team<W>;
  constexpr int kTeams = kPickThreads / (32 * W), kSize = 32 * W;
  __shared__ typename TeamW::Shared shared[kTeams];
  follow();
  const int row = blockIdx.x * kTeams + (W > 1 ? 0 : threadIdx.x >> 5);
  if (row >= a.B * a.lists * a.c.kv_heads) return;
  TeamW team(shared[W > 1 ? 0 : threadIdx.x >> 5], W > 1 ? threadIdx.x : threadIdx.x & 31);
  const int tid = team.thread, lane = tid & 31;
  const int bt = row / a.c.kv_heads, h = row - bt * a.c.kv_heads;
  const int b = bt / a.lists, t = bt - b * a.lists;
  const Seq q = find_seq(a, b, false);
  if (q.F < 0 || t >= q.tokens) return;
  int32_t* out = a.pages + (size_t)row * a.count;
  if (q.F <= a.count) {  // all of them
    for (int i = tid; i < a.count; i += kSize) out[i] = i < q.F ? i : -1;
    return;
  }
  const int lo = a.first, hi = q.F - a.last, want = a.count - a.first - a.last;
  const float* scores = a.scores + (size_t)row * a.stride;
  float held[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int j = i * kSize + tid;
    held[i] = j < q.F ? scores[j] : 0.0f;
  }
  // f(page, score) of every candidate that is this thread's; whole warps take
  // part, with page = -1 where a lane has none
  auto all = [&](auto f) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i * kSize >= q.F) break;
      const int j = i * kSize + tid;
      f(j >= lo && j < hi ? j : -1, held[i]);
    }
#pragma unroll 1
    for (int i = R * kSize; i < q.F; i += kSize) {
      const int j = i + tid;
      f(j >= lo && j < hi ? j : -1, j < q.F ? scores[j] : 0.0f);
    }
  };
  // What decides: pages with scores from `edge` on (above it where `open`) are
  // taken, and of the `listed` others from `near` on those that the exact scores say:
  // the list in shared memory names the taken ones, or, of many, the ones above
  // `cut` are taken and the first `ties` that equal it.
  float edge = INFINITY, near = INFINITY;
  bool open = true, many = false;
  int listed = 0, ties = 0;
  uint64_t cut = ~0ull;
  if (want > 0) {
    uint32_t least = ~0u, most = 0;
    all([&](int j, float s) {
      const uint32_t k = j < 0 ? ~0u : ordered_bits(s);
      least = k < least ? k : least;
      most = j >= 0 && k > most ? k : most;
    });
    // `want` scores are at or above `at`, or more, and then all below at + 1
    uint32_t at = team.least(least), above = team.most(most) + 1;
    bool split = false;
#pragma unroll 1
    while (!split && above - at > 1) {
      const uint32_t mid = at + (above - at) / 2;
      uint32_t n = 0;
      all([&](int j, float s) { n += j >= 0 && ordered_bits(s) >= mid; });
      n = team.sum(n);
      split = n == (uint32_t)want;
      if (n >= (uint32_t)want) at = mid;
      else above = mid;
    }
    uint32_t in = ~0u, out_key = 0;  // the lowest that is taken, the highest that is not
    all([&](int j, float s) {
      const uint32_t k = ordered_bits(s);
      if (j >= 0 && k >= at && k < in) in = k;
      if (j >= 0 && k < at && k > out_key) out_key = k;
    });
    in = team.least(in);
    out_key = split ? team.most(out_key) : in;
    const float kth = from_ordered_bits(in), next = from_ordered_bits(out_key);
    float reach_k = 0.0f, reach_q = 0.0f;
    const float* of = a.reach_k + ((size_t)b * a.c.kv_heads + h) * a.reaches;
    for (int i = lane; i * kReachPages < q.F; i += 32) reach_k = max_nan(reach_k, of[i]);
    const int first_token = a.lists > 1 ? t : 0, tokens = a.lists > 1 ? 1 : q.tokens;
    for (int i = lane; i < tokens; i += 32)
      reach_q = max_nan(reach_q, a.reach_q[((size_t)b * a.T + first_token + i) * a.c.kv_heads + h]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      reach_k = max_nan(reach_k, __shfl_xor_sync(0xffffffffu, reach_k, x));
      reach_q = max_nan(reach_q, __shfl_xor_sync(0xffffffffu, reach_q, x));
    }
    const float size = reach_q * reach_k;  // no sum of a score's terms is larger
    const float eps = (float)a.c.head_dim * 0x1p-22f * size;
    edge = kth;
    open = false;
    if (!(kth - next > 2.0f * eps)) {
      // scores within 2 eps of the last one that is taken could change places
      const bool known = size <= 0x1p100f && fabsf(kth) <= 0x1p101f;
      // sums below 2^62; a product that float32 cannot hold whole is far below 1
      const float scale = size == 0.0f ? 1.0f
                          : known && size >= 0x1p-60f ? __int_as_float((127 + 60 - ilogbf(size)) << 23) : 0.0f;
      const float sure = known ? kth + 2.0f * eps : INFINITY;
      near = known ? kth - 2.0f * eps : -INFINITY;
      uint32_t n = 0, m = 0;
      all([&](int j, float s) {
        n += j >= 0 && s > sure;
        m += j >= 0 && s >= near && s <= sure;
      });
      const int need = want - (int)team.sum(n);
      listed = (int)team.sum(m);
      many = listed > kNear;
      auto exact = [&](int j) {
        return exact_score<T>(a, b, first_token, tokens, h, cache_page(a.c, q.s, j, a.c.max_pages), scale, lane);
      };
      edge = sure;
      open = true;
      if (listed == need) {  // all of them
        edge = near;
        open = many = false;
        listed = 0;
      } else if (!many) {
        if (tid == 0) team.sh.n = 0;
        team.sync();
        all([&](int j, float s) {
          if (j >= 0 && s >= near && s <= sure) team.sh.near[atomicAdd(&team.sh.n, 1)] = j;
        });
        team.sync();
#pragma unroll 1
        for (int e = tid >> 5; e < listed; e += W) {
          const uint64_t x = exact(team.sh.near[e]);
          if (lane == 0) team.sh.exact[e] = x;
        }
        team.sync();
        // rank by score, then by place; those that stay out are marked
        bool stays = true;
        if (tid < listed) {
          const uint64_t x = team.sh.exact[tid];
          const int j = team.sh.near[tid];
          int rank = 0;
          for (int e = 0; e < listed; ++e) {
            const uint64_t y = team.sh.exact[e];
            rank += y > x || (y == x && team.sh.near[e] < j);
          }
          stays = rank < need;
        }
        team.sync();
        if (tid < listed && !stays) team.sh.near[tid] = -1;
        team.sync();
      } else {
        uint64_t* border = a.border + (size_t)row * a.stride;
        all([&](int j, float s) {
          uint32_t here = __ballot_sync(0xffffffffu, j >= 0 && s >= near && s <= sure);
          while (here) {
            const int l = __ffs(here) - 1;
            here &= here - 1;
            const int page = __shfl_sync(0xffffffffu, j, l);
            const uint64_t x = exact(page);
            if (lane == l) border[page] = x;
          }
        });
        // the need-th largest of them (each thread reads what it has written)
        uint64_t low = 0, high = ~0ull;
#pragma unroll 1
        while (high - low > 1) {
          const uint64_t mid = low + (high - low) / 2;
          uint32_t n2 = 0;
          all([&](int j, float s) {
            n2 += j >= 0 && s >= near && s <= sure && border[j] >= mid;
          });
          n2 = team.sum(n2);
          if (n2 >= (uint32_t)need) low = mid;
          else high = mid;
        }
        cut = low;
        uint32_t n2 = 0;
        all([&](int j, float s) {
          n2 += j >= 0 && s >= near && s <= sure && border[j] > cut;
        });
        ties = need - (int)team.sum(n2);
      }
    }
  }
  // the taken pages in order
  const uint64_t* border = a.border + (size_t)row * a.stride;
  int done = 0, tied = 0;
  auto write = [&](int j, float s) {
    bool take = j < lo || (j >= hi && j < q.F), tie = false;
    if (!take && j < hi) {
      take = open ? s > edge : s >= edge;
      if (!take && listed > 0 && s >= near) {
        if (many) {
          const uint64_t k = border[j];
          take = k > cut;
          tie = k == cut;
        } else {
          for (int e = 0; e < listed; ++e) take |= team.sh.near[e] == j;
        }
      }
    }
    if (many) {  // as many of those on the border as there is room for, the first ones
      const uint32_t m = __ballot_sync(0xffffffffu, tie);
      int before = tied;
      if (W > 1) {
        __syncthreads();
        if (lane == 0) team.sh.part[0][tid >> 5] = __popc(m);
        __syncthreads();
        for (int w = 0; w < W; ++w) {
          if (w < tid >> 5) before += (int)team.sh.part[0][w];
          tied += (int)team.sh.part[0][w];
        }
      } else {
        tied += __popc(m);
      }
      if (tie) take = before + __popc(m & ((1u << lane) - 1)) < ties;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    int at = done;
    if (W > 1) {
      __syncthreads();
      if (lane == 0) team.sh.part[1][tid >> 5] = __popc(m);
      __syncthreads();
      for (int w = 0; w < W; ++w) {
        if (w < tid >> 5) at += (int)team.sh.part[1][w];
        done += (int)team.sh.part[1][w];
      }
    } else {
      done += __popc(m);
    }
    at += __popc(m & ((1u << lane) - 1));
    if (take && at < a.count) out[at] = j;
  };
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (i * kSize < q.F) write(i * kSize + tid, held[i]);
#pragma unroll 1
  for (int i = R * kSize; i < q.F; i += kSize) write(i + tid, i + tid < q.F ? scores[i + tid] : 0.0f);
}

template <typename T>
cudaError_t launch_pick(const SelectArgs& a, cudaStream_t stream) {
  const int rows = a.B * a.lists * a.c.kv_heads;
  if (a.c.max_pages <= 256)
    return launch_behind(pick_pages_kernel<T, 1, 8>, (rows + 7) / 8, kPickThreads, 0, stream, a);
  return launch_behind(pick_pages_kernel<T, 8, 8>, rows, kPickThreads, 0, stream, a);
}

// Blocks for the stretches of a table: as many as it can have, unless the batch alone
// fills the GPU many times over; the blocks of short sequences end at once.
template <typename... P>
cudaError_t launch_score(void (*kernel)(P...), const SelectArgs& a, int pages, int sms, cudaStream_t stream) {
  const int stretches = (a.c.max_pages + pages * kScoreWarps - 1) / (pages * kScoreWarps);
  const int heads = a.B * a.c.kv_heads, most = (32 * sms + heads - 1) / heads;
  return launch_behind(kernel, dim3(stretches < most ? stretches : most, a.c.kv_heads, a.B), kScoreThreads, 0,
                       stream, a);
}

template <int KD>
cudaError_t launch_mma(const SelectArgs& a, int sms, cudaStream_t stream) {
  const int rows = a.T * a.group;
  return launch_score(rows <= 8 ? score_mma_kernel<1, KD> : rows <= 16 ? score_mma_kernel<2, KD> : score_mma_kernel<4, KD>,
                      a, 16, sms, stream);
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& a, int sms, cudaStream_t stream) {
  cudaError_t e;
  if (a.c.dtype == DSPARK_BF16 && a.c.head_dim % 32 == 0)
    e = a.c.head_dim == 128 ? launch_mma<4>(a, sms, stream)
        : a.c.head_dim == 64 ? launch_mma<2>(a, sms, stream) : launch_mma<0>(a, sms, stream);
  else
    e = launch_score(a.c.dtype == DSPARK_F32 ? score_ffma_kernel<float> : score_ffma_kernel<__nv_bfloat16>, a,
                     kReachPages, sms, stream);
  if (e != cudaSuccess) return e;
  return a.c.dtype == DSPARK_F32 ? launch_pick<float>(a, stream) : launch_pick<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
