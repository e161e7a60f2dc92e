// cache_append.cu -- queries and keys normalised for each head and rotated by
// their positions, and keys and values stored to the pages, in one pass.
//
// For a head's row x of D values: r = 1 / sqrt(mean(x^2) + eps), y = x r w,
// then the pairs (a, b) of the first rot_dim values turn by the position's
// angle: (a c - b s, b c + a s).  Everything is float32 and rounded once.
// Every value is read once and written once, so the pass is bound by HBM for
// prompts and by one launch's latency for single tokens.
//
// Vector kernel: a group of D * size / 16 lanes holds a row, 16 bytes a lane,
// so a warp's load is 512 contiguous bytes; the mean is a butterfly over the
// group, and the other half of a pair sits in the lane rot_dim / 2 values
// away (or in the same lane, for neighbouring pairs).  A warp stays on one
// token, so the rotation's cosines are loaded once for all its heads.  Two
// prompts of 8191 and fewer tokens, 8 x 4 heads of 128 dims, take 59 us with
// neighbouring pairs, 5.6 TB/s, 0.83 of a copy's rate, and 76.5 with pairs half a
// rotation apart, whose partners come from other lanes; one token 4.3 us a replay.
// Five blocks a multiprocessor, four in brackets, us a replay: neighbouring pairs
// 60.4 (62.0), 64 dims 34.9 (36.4), 256 dims 112.7 (116.2); half-split pairs 76.5
// (80.0), 64 dims 43.4 (45.1), 256 dims 143.4 (147.6), although five blocks' 96
// registers spill 56 to 64 bytes there; the drafts of a full batch 8.3 (9.7);
// float32, whose lanes hold half the values and spill nothing either way, 73.5
// (71.8) and with neighbouring pairs 63.0 (62.4).  Rows that do not split that way
// (other head dims than 8, 16 or 32 lanes hold, rotations that end inside a lane's
// words, unaligned tables) take the row kernel: a warp for each row, through shared
// memory, one value a load: 332 us for such prompts with heads of 96 dims (0.75
// TB/s), bound by its instructions, and 6.2 us for one token.
#include "cache.cuh"
#include "host_util.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 128;

template <typename T>
struct Word;  // 16 bytes of T as float32
template <>
struct Word<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void load(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                      __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Where a token goes.  page < 0: its keys and values are not stored.
struct Token {
  int b, t, page, slot, position;
  bool there;
};

__device__ __forceinline__ Token find_token(const AppendArgs& a, int i, bool report) {
  Token k;
  k.b = i / a.T;
  k.t = i - k.b * a.T;
  k.page = -1;
  k.slot = 0;
  k.position = a.position[i];
  const int s = cache_seq(a.c, a.seq, k.b);
  k.there = s >= 0 && (a.count == nullptr || k.t < a.count[k.b]);
  if (s < 0 && report) cache_error(a.c, kCacheErrSeq);
  if (!k.there) return k;
  const int len = a.length[k.b];
  // held pages hold at most 2^30 tokens, and t < 2^24
  if (len >= 0 && len < (1 << 30)) {
    const uint32_t i = page_of(a.c, (uint32_t)(len + k.t), k.slot);
    if (i < (uint32_t)cache_held(a.c, s)) k.page = cache_page(a.c, s, (int)i, a.c.max_pages);
  }
  if (k.page < 0 && report) cache_error(a.c, kCacheErrPage);
  if (k.position < 0 || k.position >= a.max_position) {
    k.position = -1;
    if (report) cache_error(a.c, kCacheErrPosition);
  }
  return k;
}

// Row `h` of token k: queries, then keys, then values.  Null if there is no
// such row, or nothing to store it to.
struct Row {
  const char* src;
  char* dst;
  const float* weight;
  bool rotate;
};

__device__ __forceinline__ Row find_row(const AppendArgs& a, const Token& k, int h) {
  const int Hq = a.heads, Hk = a.c.kv_heads;
  const size_t elt = dtype_bytes(a.c.dtype), row = a.c.head_dim * elt;
  const size_t token = (size_t)k.b * a.T + k.t;
  Row r{nullptr, nullptr, nullptr, false};
  if (h < Hq) {
    r.src = a.q + token * a.q_stride * elt + h * row;
    r.dst = a.q_out + (token * Hq + h) * row;
    r.weight = a.q_weight;
    r.rotate = true;
  } else if (h < Hq + 2 * Hk && k.page >= 0) {
    const bool key = h < Hq + Hk;
    const int g = h - Hq - (key ? 0 : Hk);
    r.src = key ? a.k + token * a.k_stride * elt + g * row
                : a.v + token * a.v_stride * elt + g * row;
    r.dst = static_cast<char*>(a.c.pool) +
            cache_row(a.c, 2 * a.layer + (key ? 0 : 1), k.page, g, k.slot);
    r.weight = key ? a.k_weight : nullptr;
    r.rotate = key;
  }
  return r;
}

// n floats from p, 16 (n a multiple of 4) or 8 bytes at a time.
template <int n>
__device__ __forceinline__ void load_floats(const float* p, float* x) {
  if (n % 4 == 0) {
#pragma unroll
    for (int i = 0; i < n / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x;
    x[1] = v.y;
  }
}

// kLanes lanes hold a row; a warp takes `batches` times kPer loads of a token,
// the next batch on its way while one is worked on.  The table and the weights
// are read 16 bytes at a time (one value at a time the loads of angles and
// weights, not HBM, bound the pass: 119 us for two prompts of 13k tokens), and
// the first batch is under way before the token's place is looked up (97 us
// when each warp took one batch and looked its token up first).
template <typename T, int kLanes, int kPer, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(AppendArgs a, int splits, int batches) {
  constexpr int N = Word<T>::n, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int token = w / splits, split = w - token * splits;
  if (token >= a.B * a.T) return;
  follow();
  const int sub = lane & (kLanes - 1);
  const int d0 = sub * N, half = a.rot >> 1;
  const int Hq = a.heads, Hk = a.c.kv_heads;
  constexpr int elt = sizeof(T), row = kLanes * 16;
  const char* q = a.q + (size_t)token * a.q_stride * elt + 16 * sub;
  const char* kk = a.k + (size_t)token * a.k_stride * elt + 16 * sub - Hq * row;
  const char* v = a.v + (size_t)token * a.v_stride * elt + 16 * sub - (Hq + Hk) * row;
  int h0 = split * batches * kPer * kRows + lane / kLanes;
  uint4 word[kPer];
  auto load = [&](int from, uint4 (&to)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = from + i * kRows;
      const char* src = h < Hq ? q : h < Hq + Hk ? kk : v;
      to[i] = make_uint4(0, 0, 0, 0);
      if (h < Hq + 2 * Hk) to[i] = __ldcs(reinterpret_cast<const uint4*>(src + h * row));
    }
  };
  load(h0, word);
  const Token k = find_token(a, token, lane == 0 && split == 0);
  if (!k.there) return;
  // the angle of each of the lane's values; the sine carries the sign
  float cs[N], sn[N];
  int partner = lane;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
  }
  const bool turn = k.position >= 0 && d0 < a.rot;  // all the lane's values or none
  if (turn) {
    const float* table = a.cos_sin + (size_t)k.position * a.rot;
    if (!kInterleaved) {
      const bool low = d0 < half;
      partner = low ? lane + half / N : lane - half / N;
      load_floats<N>(table + (low ? d0 : d0 - half), cs);
      load_floats<N>(table + (low ? d0 + half : d0), sn);
      if (low)
#pragma unroll
        for (int e = 0; e < N; ++e) sn[e] = -sn[e];
    } else {
      float c2[N / 2], s2[N / 2];
      load_floats<N / 2>(table + (d0 >> 1), c2);
      load_floats<N / 2>(table + half + (d0 >> 1), s2);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        cs[e] = c2[e >> 1];
        sn[e] = e & 1 ? s2[e >> 1] : -s2[e >> 1];
      }
    }
  }
  const bool norm = a.q_weight || a.k_weight;
  float wq[N], wk[N];
  if (a.q_weight) load_floats<N>(a.q_weight + d0, wq);
  if (a.k_weight) load_floats<N>(a.k_weight + d0, wk);
  auto two = [](const float (&f)[N], int e) { return pair(f[2 * e], f[2 * e + 1]); };
  char* q_out = a.q_out + (size_t)token * Hq * row + 16 * sub;
  const size_t step = (size_t)a.c.page_size * row;  // between a page's heads
  char* k_out = static_cast<char*>(a.c.pool) +
                cache_row(a.c, 2 * a.layer, k.page < 0 ? 0 : k.page, 0, k.slot) + 16 * sub;
  char* v_out = k_out + cache_row(a.c, 1, 0, 0, 0);
  for (int batch = 0; batch < batches; ++batch) {
    uint4 ahead[kPer];
    if (kPer > 1 && batch + 1 < batches) load(h0 + kPer * kRows, ahead);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = h0 + i * kRows;
      const bool is_q = h < Hq, is_k = !is_q && h < Hq + Hk;
      if (h - lane / kLanes >= Hq + Hk) {  // values only
        if (h < Hq + 2 * Hk && k.page >= 0)
          *reinterpret_cast<uint4*>(v_out + (h - Hq - Hk) * step) = word[i];
        continue;
      }
      float x[N];
      uint64_t x2[N / 2];
      Word<T>::load(word[i], x);
#pragma unroll
      for (int e = 0; e < N / 2; ++e) x2[e] = two(x, e);
      if (norm) {  // the butterfly is the whole warp's
        uint64_t sum2 = 0;
#pragma unroll
        for (int e = 0; e < N / 2; ++e) sum2 = fma2(x2[e], x2[e], sum2);
        const float2 halves = unpair(sum2);
        float sum = halves.x + halves.y;
#pragma unroll
        for (int m = kLanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float r = rsqrtf(sum * (1.0f / (kLanes * N)) + a.eps);
        if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
#pragma unroll
          for (int e = 0; e < N / 2; ++e)
            x2[e] = mul2(mul2(x2[e], pair(r, r)), is_q ? two(wq, e) : two(wk, e));
        }
      }
      // a value that is not turned keeps its bits (0 * infinity is no 0)
      uint64_t y2[N / 2];
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 f = unpair(x2[e]);
        y2[e] = kInterleaved ? pair(f.y, f.x)
                             : pair(__shfl_sync(0xffffffffu, f.x, partner),
                                    __shfl_sync(0xffffffffu, f.y, partner));
      }
      if (turn) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
          x2[e] = fma2(x2[e], two(cs, e), mul2(y2[e], two(sn, e)));
      }
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 f = unpair(x2[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(q_out + h * row) = Word<T>::store(x);
      } else if (k.page >= 0) {
        if (is_k) *reinterpret_cast<uint4*>(k_out + (h - Hq) * step) = Word<T>::store(x);
        else if (h < Hq + 2 * Hk) *reinterpret_cast<uint4*>(v_out + (h - Hq - Hk) * step) = word[i];
      }
    }
    if (kPer > 1) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) word[i] = ahead[i];
    }
    h0 += kPer * kRows;
  }
}

// A warp for each row, any head_dim and rot_dim.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_row_kernel(AppendArgs a) {
  __shared__ float buf[kThreads / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = a.heads + 2 * a.c.kv_heads, D = a.c.head_dim;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + warp;
  const int token = (int)(w / rows), h = (int)(w - (long long)token * rows);
  if (token >= a.B * a.T) return;
  follow();
  const Token k = find_token(a, token, lane == 0 && h == 0);
  if (!k.there) return;
  const Row r = find_row(a, k, h);
  if (!r.src) return;
  const T* src = reinterpret_cast<const T*>(r.src);
  T* dst = reinterpret_cast<T*>(r.dst);
  if (!r.rotate) {  // values: the bits
    for (int d = lane; d < D; d += 32) dst[d] = src[d];
    return;
  }
  float sum = 0.0f;
  for (int d = lane; d < D; d += 32) {
    const float x = to_float(src[d]);
    buf[warp][d] = x;
    sum = fmaf(x, x, sum);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const float rs = r.weight ? rsqrtf(sum / (float)D + a.eps) : 1.0f;
  __syncwarp();
  const int half = a.rot >> 1;
  const float* table = a.cos_sin + (size_t)(k.position < 0 ? 0 : k.position) * a.rot;
  for (int d = lane; d < D; d += 32) {
    float x = buf[warp][d];
    if (r.weight) x = x * rs * r.weight[d];
    if (k.position >= 0 && d < a.rot) {
      const int i = a.interleaved ? d >> 1 : d < half ? d : d - half;
      const bool low = a.interleaved ? !(d & 1) : d < half;
      const int o = a.interleaved ? d ^ 1 : low ? d + half : d - half;
      float y = buf[warp][o];
      if (r.weight) y = y * rs * r.weight[o];
      const float sn = table[half + i];
      x = fmaf(x, table[i], low ? -y * sn : y * sn);
    }
    put(dst + d, x);
  }
}

template <typename T, int kLanes>
cudaError_t launch_lanes(const AppendArgs& a, cudaStream_t stream) {
  const int rows = a.heads + 2 * a.c.kv_heads;
  const long long tokens = (long long)a.B * a.T;
  // rows of a warp's load, and loads of a token
  const int per_warp = 32 / kLanes, loads = (rows + per_warp - 1) / per_warp;
  // Four loads a batch, and a whole token a warp, as far as that leaves every
  // multiprocessor 16 warps; fewer tokens than that are bound by latency.
  const long long enough = 16LL * sm_count();
  const bool many = tokens * ((loads + 3) / 4) >= enough;
  const int all = many ? (loads + 3) / 4 : loads;  // batches of a token
  int splits = all;
  while (many && splits > 1 && tokens * (splits / 2) >= enough) splits = (splits + 1) / 2;
  const int batches = (all + splits - 1) / splits;
  if (tokens * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned blocks = (unsigned)((tokens * splits + kThreads / 32 - 1) / (kThreads / 32));
  const auto kernel = many ? (a.interleaved ? append_kernel<T, kLanes, 4, true>
                                            : append_kernel<T, kLanes, 4, false>)
                           : (a.interleaved ? append_kernel<T, kLanes, 1, true>
                                            : append_kernel<T, kLanes, 1, false>);
  return launch_behind(kernel, blocks, kThreads, 0, stream, a, splits, batches);
}

template <typename T>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int N = Word<T>::n;
  // a lane's values turn together and read whole words of the table
  const bool whole =
      (a.interleaved ? a.rot % N == 0 && (a.rot >> 1) % (N / 2) == 0 : (a.rot >> 1) % N == 0) &&
      aligned_to(a.cos_sin, 16) && aligned_to(a.q_weight, 16) && aligned_to(a.k_weight, 16);
  if (whole && a.c.head_dim == 8 * N) return launch_lanes<T, 8>(a, stream);
  if (whole && a.c.head_dim == 16 * N) return launch_lanes<T, 16>(a, stream);
  if (whole && a.c.head_dim == 32 * N) return launch_lanes<T, 32>(a, stream);
  const long long blocks =
      ((long long)a.B * a.T * (a.heads + 2 * a.c.kv_heads) + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_behind(append_row_kernel<T>, (unsigned)blocks, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  return a.c.dtype == DSPARK_F32 ? launch<float>(a, stream)
                                 : launch<__nv_bfloat16>(a, stream);
}

}  // namespace dspark
