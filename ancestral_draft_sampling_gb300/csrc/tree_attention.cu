// tree_attention.cu -- attention of drafted tokens over the paged cache on
// the FFMA units (float32, and the shapes that the tensor-core kernel does
// not take), and the merge of partial results.
//
// One pass over a unit's keys with the running maximum m and sum l of each
// row: for a tile, s = scale q.k, m' = max(m, max s), p = exp(s - m'),
// l' = l e^(m - m') + sum p, o' = o e^(m - m') + p v.  All of it is float32.
//
// Scores are in units of log2, so that a weight is one ex2.
//
// Sixteen warps share a tile of 64 keys (32 where head_dim is above 128) in
// shared memory.  A warp holds four rows (eight warps with eight rows each where
// there are enough), and two to sixteen groups of warps take the same rows and
// part of the keys each, with statistics of their own (a row's maximum is the
// warp's; its sum stays spread over the lanes); the groups are joined at the
// unit's end.  The next tile, of whatever unit, is copied (cp.async) while one is
// worked on, and the pages of the one behind it are looked up.  Products are
// packed, two a lane.  For 8 x 8 tokens, 4 x 8 heads, 2000 keys of 128 dims: 81
// us, where the FFMA units' rate allows 19.  A tile takes some 11000 cycles:
// scores 3500 and sums 3500, of which the products are 2000 each and the rest
// loads from shared memory (a load that all lanes share costs as much as one of
// their own of the same width), softmax 1500, the copies' issue 1850.  Loads one
// step ahead, copies of whole rows in bulk and a lane for each key were slower.
// The variants of four rows a warp have 16 warps a block and so 128 registers a
// thread, and spill 200 to 480 bytes of them; those of eight rows have 255 and
// spill nothing up to 128 dims (24 to 72 bytes above).  bfloat16 runs here where
// the tensor cores' kernel does not take the shape: 88 x 8 tokens, 8 x 4 heads,
// up to 2000 keys take 778 us with 96 dims, 806 with 128 dims and pages of 12
// rows (95 on the tensor cores with pages of 64), 1582 with 256 dims.
#include "dspark_common.cuh"
#include "host_util.cuh"
#include "sm100_ptx.cuh"
#include "tree_attention.cuh"

namespace dspark {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 32;  // of a unit

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

// Two partial sums of a dot product.
__device__ __forceinline__ uint64_t dot4(float4 a, float4 b, uint64_t c) {
  return fma2(pair(a.z, a.w), pair(b.z, b.w), fma2(pair(a.x, a.y), pair(b.x, b.y), c));
}

// 16 bytes to shared memory, or zeros where `there` is false.
__device__ __forceinline__ void copy16(void* to, const void* from, bool there) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(to)), "l"(from),
               "r"(n)
               : "memory");
}

// Shared memory of a block, in bytes.
template <typename T, int ND, int RW>
struct Tiles {
  static constexpr int kWarps = 2 * kRows / RW, kThreads = 32 * kWarps;
  static constexpr int kTile = ND == 1 ? 64 : 32;  // keys
  int D;
  __host__ __device__ int pad() const { return D + 16 / (int)sizeof(T); }  // rows on different banks
  __host__ __device__ int key_bytes() const { return kTile * pad() * (int)sizeof(T); }
  __host__ __device__ int value_bytes() const { return kTile * D * (int)sizeof(T); }
  __host__ __device__ int stage() const { return key_bytes() + value_bytes(); }
  // the queries, and at a unit's end the parts that groups leave each other
  __host__ __device__ int q_at() const { return 2 * stage(); }
  __host__ __device__ int p_at() const { return q_at() + kRows * (D + 4) * 4; }
  __host__ __device__ int where_at() const { return p_at() + kWarps * (kTile / 2) * RW * 4; }
  __host__ __device__ int total() const { return where_at() + 2 * kTile * 8; }
};

// A tile of the block's line, one ahead of the work.
struct NextTile {
  TreeWalk w;
  int i;      // within the unit
  bool some;
  __device__ __forceinline__ void step(const TreeArgs& a) {
    if (++i < w.n) return;
    i = 0;
    some = w.next(a);
  }
};

// ND: chunks of 128 dims that a warp's four each cover (1: D <= 128, 2: D <=
// 256); halves: half a warp covers them (D <= 64), so the other half of it takes
// the sums over every other key (60 tokens over 1500 keys of 64: 116 -> 96 us).
template <typename T, int ND, bool halves, int RW>
__global__ void __launch_bounds__(Tiles<T, ND, RW>::kThreads)
    tree_ffma_kernel(const __grid_constant__ TreeArgs a, int row_groups) {
  using L = Tiles<T, ND, RW>;
  constexpr int kTile = L::kTile, kWarps = L::kWarps, kThreads = L::kThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ TreeShare share;
  __shared__ uchar2 row_of[kRows];  // a row's token and head
  const int D = a.c.head_dim, DP = D + 4;
  const L layout{D};
  const int pad = layout.pad(), words = D * (int)sizeof(T) / 16;
  float* qs = reinterpret_cast<float*>(smem + layout.q_at());  // [kRows][DP], scaled
  long long* where = reinterpret_cast<long long*>(smem + layout.where_at());  // [2][kTile]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* pw = reinterpret_cast<float*>(smem + layout.p_at()) + warp * (kTile / 2) * RW;  // weights
  // the warp's rows and keys
  const int key_groups = kWarps / row_groups, rg = warp & (row_groups - 1), kg = warp / row_groups;
  const int keys = kTile / key_groups, key0 = kg * keys;
  // of a warp's keys, four to a lane while scores are made, one after that
  const int key_lanes = keys / 4, key_lane = lane & (key_lanes - 1);
  const int key_shift = 31 - __clz(key_lanes), segment = lane >> key_shift;
  const int share_of = 4 * ((D / 4 * key_lanes + 31) / 32);
  const int dim0 = segment * share_of, dim1 = dim0 + share_of < D ? dim0 + share_of : D;
  const int lane_key = key_lane + key_lanes * (2 * (segment & 1) + ((segment >> 1) & 1));
  auto holder = [&](int j) {  // the lane of key j
    const int x = j >> key_shift;
    return ((x >> 1) + 2 * (x & 1)) * key_lanes + (j & (key_lanes - 1));
  };
  // of the sums a lane has four dims, of every key or, where half a warp covers
  // the head, of every other
  const int dim = 4 * (halves ? lane & 15 : lane), odd_key = halves ? lane >> 4 : 0;
  constexpr int key_step = halves ? 2 : 1;
  const T* q = static_cast<const T*>(a.q);
  const char* pool = static_cast<const char*>(a.c.pool);
  if (threadIdx.x < kRows) {
    const uint32_t t = threadIdx.x / (uint32_t)a.group;
    row_of[threadIdx.x] = make_uchar2(t, threadIdx.x - t * a.group);
  }
  const float c = a.scale * 1.4426950408889634f;
  follow();
  tree_start(a, share);
  NextTile ahead{share.walk, 0, share.walk.n > 0};
  TreeWalk w = share.walk;

  // Where a tile's keys lie (bytes from the start of the pool, -1: zeros), a
  // key a thread: the page is loaded first and used when the tile before is
  // done.
  int look_page = -1, look_slot = 0, look_head = 0;
  bool look_there = false;
  auto look = [&]() {
    look_there = false;
    if (threadIdx.x < kTile && ahead.some) {
      const int j = ((ahead.w.q.lo + ahead.w.first + ahead.i) * kTile) + threadIdx.x;
      look_head = ahead.w.h;
      look_there = j < ahead.w.q.len + ahead.w.q.cnt;
      if (look_there)
        look_page = a.c.block_table[(size_t)ahead.w.q.s * a.c.max_pages +
                                    page_of(a.c, (uint32_t)j, look_slot)];
    }
  };
  auto found = [&](int buffer) {
    if (threadIdx.x < kTile) {
      long long at = -1;
      if (look_there) {
        if (look_page >= 0 && look_page < a.c.num_pages)
          at = (long long)cache_row(a.c, 2 * a.layer, look_page, look_head, look_slot);
        else
          cache_error(a.c, kCacheErrPage);
      }
      where[buffer * kTile + threadIdx.x] = at;
    }
  };
  const size_t to_values = cache_row(a.c, 1, 0, 0, 0);
  const int row_step = kThreads / words, word_step = kThreads - row_step * words;
  const int copy_row = (int)threadIdx.x / words, copy_word = (int)threadIdx.x - copy_row * words;
  auto copy = [&](int buffer) {
    uint8_t* stage = smem + buffer * layout.stage();
    int r = copy_row, d = copy_word;
#pragma unroll 2
    for (int i = threadIdx.x; i < 2 * kTile * words; i += kThreads) {
      const bool value = r >= kTile;
      const int key = value ? r - kTile : r;
      const long long at = where[buffer * kTile + key];
      uint8_t* to = value ? stage + layout.key_bytes() + key * D * (int)sizeof(T)
                          : stage + key * pad * (int)sizeof(T);
      copy16(to + 16 * d, pool + (at < 0 ? 0 : at + (value ? to_values : 0)) + 16 * d, at >= 0);
      r += row_step;
      d += word_step;
      if (d >= words) {
        d -= words;
        ++r;
      }
    }
  };
  // the first tile, and where the second lies
  look();
  found(0);
  __syncthreads();
  if (ahead.some) {
    copy(0);
    ahead.step(a);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  look();
  found(1);
  int n = 0;  // tiles worked on
  bool is_first = true;
  for (bool some = w.n > 0; some; some = w.next(a)) {
    const int t0 = w.rt * a.row_tokens;
    const int rows = (w.q.cnt - t0 < a.row_tokens ? w.q.cnt - t0 : a.row_tokens) * a.group;
    const int head0 = w.h * a.group;
    __syncthreads();  // the last unit's queries are used up
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int r = (int)((uint32_t)i / (uint32_t)(D / 4)), d = (i - r * (D / 4)) * 4;
      const int t = t0 + row_of[r].x, g = row_of[r].y;
      const float4 x = load4(q + (((size_t)w.b * a.T + t) * a.heads + head0 + g) * D + d);
      *reinterpret_cast<float4*>(qs + r * DP + d) =
          make_float4(x.x * c, x.y * c, x.z * c, x.w * c);
    }
    float m[RW], l[RW];
    uint64_t o[RW][ND][2];
    uint64_t bits[RW];
    int lo[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = rg * RW + i;
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int x = 0; x < ND; ++x) o[i][x][0] = o[i][x][1] = 0;
      bits[i] = 0;
      lo[i] = w.q.len;
      if (r < rows) {
        const int t = t0 + row_of[r].x;
        bits[i] = tree_mask(a, w.b, t, w.q.cnt);
        lo[i] = tree_window_lo(a, w.b, t, w.q.len);
      }
    }
    const int total = w.q.len + w.q.cnt;
    const bool busy = rg * RW < rows;
#pragma unroll 1
    for (int tile = 0; tile < w.n; ++tile, ++n) {
      const int j0 = (w.q.lo + w.first + tile) * kTile;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // the tile is there, and the one before it is used up
      if (ahead.some) {
        copy((n + 1) & 1);
        ahead.step(a);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      look();
      if (!busy) {
        found(n & 1);
        continue;
      }
      const T* ks = reinterpret_cast<const T*>(smem + (n & 1) * layout.stage());
      const T* vs = reinterpret_cast<const T*>(smem + (n & 1) * layout.stage() + layout.key_bytes());
      // Scores: a lane has four keys and a stretch of the dims, 8 loads from
      // shared memory for 16 products of four (a key a lane over all dims takes
      // 5 for 4, and single tokens over 4000 keys take 119 us instead of 80).
      // The lanes of the same keys then add up and keep a key each.
      uint64_t s2[RW][4];
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) s2[i][x] = 0;
      const float* qr = qs + rg * RW * DP;
      const T* kr = ks + (key0 + key_lane) * pad;
#pragma unroll 1
      for (int d = dim0; d < dim1; d += 4) {
        float4 x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = load4(kr + y * key_lanes * pad + d);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float4 y = load4(qr + i * DP + d);
#pragma unroll
          for (int z = 0; z < 4; ++z) s2[i][z] = dot4(y, x[z], s2[i][z]);
        }
      }
      __syncwarp();
      float s[RW];
      {
        const bool odd = segment & 1, odd2 = segment & 2;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          float v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 y = unpair(s2[i][x]);
            v[x] = y.x + y.y;
          }
          const float a0 = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[2], key_lanes);
          const float a1 = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[3], key_lanes);
          const float b0 = (odd ? v[2] : v[0]) + a0, b1 = (odd ? v[3] : v[1]) + a1;
          const float c0 = __shfl_xor_sync(0xffffffffu, odd2 ? b0 : b1, 2 * key_lanes);
          s[i] = (odd2 ? b1 : b0) + c0;
        }
#pragma unroll 1
        for (int x = 4 * key_lanes; x < 32; x *= 2)
#pragma unroll
          for (int i = 0; i < RW; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
      }
      const int j = j0 + key0 + lane_key;
      const uint32_t full = keys >= 32 ? ~0u : (1u << keys) - 1;
      uint32_t seen[RW];  // the warp's keys that the row sees (bit l: lane l's)
      bool all = true;
      float now[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const bool see = lane < keys && (j < w.q.len ? j >= lo[i]
                                                     : j < total && ((bits[i] >> (j - w.q.len)) & 1));
        seen[i] = __ballot_sync(0xffffffffu, see);
        all &= seen[i] == full;
        if (!see) s[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < RW; ++i)  // a NaN is no maximum
        now[i] = fmaxf(m[i], from_ordered_bits(__reduce_max_sync(
                                 0xffffffffu, ordered_bits(s[i] == s[i] ? s[i] : -INFINITY))));
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float keep = m[i] == now[i] ? 1.0f : ex2(m[i] - now[i]);
        const float p = ((seen[i] >> lane) & 1) && s[i] != -INFINITY ? ex2(s[i] - now[i]) : 0.0f;
        l[i] = l[i] * keep + p;  // the lane's keys
        m[i] = now[i];
#pragma unroll
        for (int x = 0; x < ND; ++x) {
          o[i][x][0] = mul2(o[i][x][0], pair(keep, keep));
          o[i][x][1] = mul2(o[i][x][1], pair(keep, keep));
        }
        if (lane < keys) pw[lane_key * RW + i] = p;
      }
      __syncwarp();
      auto add = [&](int j, bool every) {
        float p[RW];
#pragma unroll
        for (int i = 0; i < RW; i += 4) {
          const float4 x = load4(pw + j * RW + i);
          p[i] = x.x;
          p[i + 1] = x.y;
          p[i + 2] = x.z;
          p[i + 3] = x.w;
        }
#pragma unroll
        for (int x = 0; x < ND; ++x) {
          const int d = x * 128 + dim;
          if (d < D) {
            const float4 v = load4(vs + (key0 + j) * D + d);
            const uint64_t v0 = pair(v.x, v.y), v1 = pair(v.z, v.w);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
              if (!every && !((seen[i] >> holder(j)) & 1)) continue;
              const uint64_t pi = pair(p[i], p[i]);
              o[i][x][0] = fma2(pi, v0, o[i][x][0]);
              o[i][x][1] = fma2(pi, v1, o[i][x][1]);
            }
          }
        }
      };
      if (all) {
#pragma unroll 4
        for (int j = 0; j < keys; j += key_step) add(j + odd_key, true);
      } else {  // a key that a row does not see is left out, whatever its values hold
#pragma unroll 1
        for (int j = 0; j < keys; j += key_step) add(j + odd_key, false);
      }
      __syncwarp();
      found(n & 1);
    }
    if (halves) {
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          o[i][0][x] = add2(o[i][0][x], __shfl_xor_sync(0xffffffffu, o[i][0][x], 16));
    }
    // the lanes' sums
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    const int slot = 2 * blockIdx.x + (is_first ? 0 : 1);
    is_first = false;
    {  // the groups' parts, one after the other into the first group's
#pragma unroll 1
      for (int g = 1; g < key_groups; ++g) {
        __syncthreads();
        if (kg == g && busy) {
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            float* at = qs + (rg * RW + i) * DP;
#pragma unroll
            for (int x = 0; x < ND; ++x) {
              const int d = x * 128 + dim;
              if (d < D) {
                *reinterpret_cast<uint64_t*>(at + d) = o[i][x][0];
                *reinterpret_cast<uint64_t*>(at + d + 2) = o[i][x][1];
              }
            }
            if (lane == 0) {
              at[D] = m[i];
              at[D + 1] = l[i];
            }
          }
        }
        __syncthreads();
        if (kg == 0 && busy) {
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const float* at = qs + (rg * RW + i) * DP;
            const float om = at[D], now = fmaxf(m[i], om);
            const float f = m[i] == now ? 1.0f : ex2(m[i] - now);
            const float g2 = om == now ? 1.0f : ex2(om - now);
            l[i] = l[i] * f + at[D + 1] * g2;
            m[i] = now;
#pragma unroll
            for (int x = 0; x < ND; ++x) {
              const int d = x * 128 + dim;
              if (d < D) {
                const uint64_t gg = pair(g2, g2), ff = pair(f, f);
                o[i][x][0] = fma2(*reinterpret_cast<const uint64_t*>(at + d), gg, mul2(o[i][x][0], ff));
                o[i][x][1] = fma2(*reinterpret_cast<const uint64_t*>(at + d + 2), gg, mul2(o[i][x][1], ff));
              }
            }
          }
        }
      }
    }
    if (kg > 0) continue;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = rg * RW + i;
      if (r >= rows) break;
      const int t = t0 + row_of[r].x, g = row_of[r].y;
      const size_t row = ((size_t)w.b * a.T + t) * a.heads + head0 + g;
      const float inv = w.whole ? (l[i] == 0.0f ? 0.0f : 1.0f / l[i]) : 1.0f;
#pragma unroll
      for (int x = 0; x < ND; ++x) {
        const int d = x * 128 + dim;
        if (d >= D) continue;
        const float2 x0 = unpair(o[i][x][0]), x1 = unpair(o[i][x][1]);
        const float4 y = make_float4(x0.x * inv, x0.y * inv, x1.x * inv, x1.y * inv);
        if (w.whole) put4(static_cast<T*>(a.out) + row * D + d, y);
        else put4(tree_part(a, slot) + (size_t)r * D + d, y);
      }
      if (lane == 0) {
        if (!w.whole) {
          float* st = tree_part_stats(a, slot) + 2 * r;
          st[0] = m[i];
          st[1] = l[i];
        } else if (a.lse) {
          a.lse[row] = l[i] == 0.0f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // behind the work, so that the first tile does not wait for it
  if (threadIdx.x == 0) tree_describe(a, share.walk);
}

// Joins the partial results of the units that several blocks worked on: o =
// sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over the unit's blocks c in
// order, M the largest m_c.  Units of few rows are bound by latency: a warp for
// each row, the loads of eight parts in flight together.
constexpr int kMergeWarps = 4;

template <typename T, int ND>
__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kBatch = 8;
  follow();
  const TreeJoin j = a.join[blockIdx.x + 1];  // nothing cuts the line's start
  const int lane = threadIdx.x & 31, D = a.c.head_dim;
  const uint32_t r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if ((int)r >= j.rows) return;
  const int parts = j.last - j.first + 1;
  auto slot_of = [&](int p) { return p == 0 ? j.slot : 2 * (j.first + p); };
  auto stats = [&](int p) {
    if (p >= parts) return make_float2(-INFINITY, 0.0f);
    return *reinterpret_cast<const float2*>(tree_part_stats(a, slot_of(p)) + 2 * r);
  };
  float4 x[kBatch][ND];
  auto load_parts = [&](int p) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const float* part = tree_part(a, slot_of(p + q)) + (size_t)r * D;
#pragma unroll
      for (int k = 0; k < ND; ++k) {
        const int d = k * 128 + lane * 4;
        x[q][k] = make_float4(0, 0, 0, 0);
        if (p + q < parts && d < D) x[q][k] = load4(part + d);
      }
    }
  };
  float2 st = stats(lane);
  load_parts(0);  // under way while the weights are made
  float M = st.x, L = 0.0f;
  float4 o[ND];
#pragma unroll
  for (int k = 0; k < ND; ++k) o[k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int p = lane + 32; p < parts; p += 32) M = fmaxf(M, stats(p).x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
#pragma unroll 1
  for (int p0 = 0; p0 < parts; p0 += 32) {
    const int n = parts - p0 < 32 ? parts - p0 : 32;
    if (p0 > 0) st = stats(p0 + lane);
    // a part that saw nothing weighs nothing
    const float w = M == -INFINITY ? 0.0f : st.x == M ? 1.0f : exp2f(st.x - M), lw = w * st.y;
#pragma unroll 1
    for (int p = 0; p < n; p += kBatch) {
      if (p0 + p > 0) load_parts(p0 + p);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (p + q >= n) break;
        const float wq = __shfl_sync(0xffffffffu, w, p + q);
        L += __shfl_sync(0xffffffffu, lw, p + q);
#pragma unroll
        for (int k = 0; k < ND; ++k) {
          o[k].x = fmaf(wq, x[q][k].x, o[k].x);
          o[k].y = fmaf(wq, x[q][k].y, o[k].y);
          o[k].z = fmaf(wq, x[q][k].z, o[k].z);
          o[k].w = fmaf(wq, x[q][k].w, o[k].w);
        }
      }
    }
  }
  const uint32_t t = r / (uint32_t)a.group;
  const size_t row = ((size_t)j.b * a.T + j.t0 + t) * a.heads + j.h * a.group + (r - t * a.group);
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

// The same for units of many rows, several waves of warps whose instructions
// bound it: a warp for four rows, with a lane for each row of eight parts'
// statistics and for what is done once a row, and the loads of two parts in
// flight (8 trees of 61 tokens: 15 us with a row's work done by all lanes, 9
// so).  Joining in the attention's blocks, by the one of a unit that comes
// last, instead of this launch took 4 us more for one request and 20 for wide
// trees.
template <typename T, int ND>
__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_rows_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kBatch = 2;
  follow();
  const TreeJoin j = a.join[blockIdx.x + 1];
  const int lane = threadIdx.x & 31, D = a.c.head_dim, sub = lane >> 2;
  const int r0 = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * 4;
  if (r0 >= j.rows) return;
  const int parts = j.last - j.first + 1, mine = r0 + (lane & 3);
  auto slot_of = [&](int p) { return p == 0 ? j.slot : 2 * (j.first + p); };
  auto stats = [&](int p) {
    if (p >= parts || mine >= j.rows) return make_float2(-INFINITY, 0.0f);
    return *reinterpret_cast<const float2*>(tree_part_stats(a, slot_of(p)) + 2 * mine);
  };
  float4 x[kBatch][4][ND];
  auto load_parts = [&](int p) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const float* part = tree_part(a, slot_of(p + q)) + (size_t)r0 * D + lane * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < ND; ++k) {
          x[q][i][k] = make_float4(0, 0, 0, 0);
          if (p + q < parts && k * 128 + lane * 4 < D && r0 + i < j.rows)
            x[q][i][k] = load4(part + i * D + k * 128);
        }
    }
  };
  float2 st = stats(sub);
  load_parts(0);  // under way while the weights are made
  float M = st.x;
#pragma unroll 1
  for (int p = sub + 8; p < parts; p += 8) M = fmaxf(M, stats(p).x);
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float L = 0.0f;
  float4 o[4][ND];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < ND; ++k) o[i][k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
  for (int p0 = 0; p0 < parts; p0 += 8) {
    const int n = parts - p0 < 8 ? parts - p0 : 8;
    if (p0 > 0) st = stats(p0 + sub);
    // a part that saw nothing weighs nothing
    const float w = M == -INFINITY ? 0.0f : st.x == M ? 1.0f : exp2f(st.x - M);
    L += w * st.y;
#pragma unroll 1
    for (int p = 0; p < n; p += kBatch) {
      if (p0 + p > 0) load_parts(p0 + p);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (p + q >= n) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, (p + q) * 4 + i);
#pragma unroll
          for (int k = 0; k < ND; ++k) {
            o[i][k].x = fmaf(wi, x[q][i][k].x, o[i][k].x);
            o[i][k].y = fmaf(wi, x[q][i][k].y, o[i][k].y);
            o[i][k].z = fmaf(wi, x[q][i][k].z, o[i][k].z);
            o[i][k].w = fmaf(wi, x[q][i][k].w, o[i][k].w);
          }
        }
      }
    }
  }
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
  const uint32_t t = (uint32_t)mine / (uint32_t)a.group;
  const size_t row =
      ((size_t)j.b * a.T + j.t0 + t) * a.heads + j.h * a.group + (mine - t * a.group);
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  if (lane < 4 && mine < j.rows && a.lse)
    a.lse[row] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = __shfl_sync(0xffffffffu, inv, i);
    const size_t to = __shfl_sync(0xffffffffu, row, i);
    if (r0 + i >= j.rows) break;
#pragma unroll
    for (int k = 0; k < ND; ++k) {
      const int d = k * 128 + lane * 4;
      if (d < D)
        put4(static_cast<T*>(a.out) + to * D + d,
             make_float4(o[i][k].x * f, o[i][k].y * f, o[i][k].z * f, o[i][k].w * f));
    }
  }
}

template <typename T, int ND, bool halves, int RW>
cudaError_t launch_ffma(TreeArgs& a, int sms, cudaStream_t stream) {
  using L = Tiles<T, ND, RW>;
  const cudaError_t e =
      cudaFuncSetAttribute(tree_ffma_kernel<T, ND, halves, RW>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, L{ND * 128}.total());
  if (e != cudaSuccess) return e;
  a.tile_shift = L::kTile == 64 ? 6 : 5;
  a.row_tokens = kRows / a.group;
  a.row_tiles = (a.T + a.row_tokens - 1) / a.row_tokens;
  a.slot_rows = (a.T < a.row_tokens ? a.T : a.row_tokens) * a.group;
  a.blocks = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
  // warps side by side over the rows that a unit has; the rest share the keys
  int groups = RW == 4 ? ND : 1;  // at least four keys a warp
  while (groups < kRows / RW && groups * RW < a.slot_rows) groups *= 2;
  return launch_behind(tree_ffma_kernel<T, ND, halves, RW>, a.blocks, L::kThreads, L{a.c.head_dim}.total(),
                       stream, a, groups);
}

template <typename T, int RW>
cudaError_t launch_ffma_dims(TreeArgs& a, int sms, cudaStream_t stream) {
  if (a.c.head_dim > 128) return launch_ffma<T, 2, false, RW>(a, sms, stream);
  return a.c.head_dim > 64 ? launch_ffma<T, 1, false, RW>(a, sms, stream)
                           : launch_ffma<T, 1, true, RW>(a, sms, stream);
}

// Eight rows a warp read keys and values half as often from shared memory, but
// leave two warps a scheduler: 81 us against 83 for 8 x 8 tokens with 4 heads
// each, 90 against 96 for 60 tokens, 82 against 78 for 3 tokens with 6.
template <typename T>
cudaError_t launch_ffma_rows(TreeArgs& a, int sms, cudaStream_t stream) {
  return a.T * a.group > 24 ? launch_ffma_dims<T, 8>(a, sms, stream)
                            : launch_ffma_dims<T, 4>(a, sms, stream);
}

}  // namespace

cudaError_t launch_tree_ffma(TreeArgs& a, int sms, cudaStream_t stream) {
  return a.c.dtype == DSPARK_F32 ? launch_ffma_rows<float>(a, sms, stream)
                                 : launch_ffma_rows<__nv_bfloat16>(a, sms, stream);
}

cudaError_t launch_tree_merge(const TreeArgs& a, cudaStream_t stream) {
  if (a.blocks < 2) return cudaSuccess;
  // Rows of a unit from which on a warp takes four.  A replay of the attention of
  // 8 requests with 4000 keys of 128 dims, a row a warp against four: 64 rows 27.4
  // and 28.1 us, 72 rows 28.7 and 28.8, 96 rows 30.3 and 28.8, 128 rows 33.2 and
  // 31.0, 488 rows 67.9 and 61.5; of 64 dims: 32 rows 21.9 and 22.6, 64 rows alike,
  // 96 rows 26.7 and 24.7.
  const bool wide = a.c.head_dim > 128, many = a.slot_rows > 64;
  const int rows = kMergeWarps * (many ? 4 : 1);
  const dim3 grid(a.blocks - 1, (a.slot_rows + rows - 1) / rows);
  const auto pick = [&](auto zero) {
    using T = decltype(zero);
    return many ? (wide ? tree_merge_rows_kernel<T, 2> : tree_merge_rows_kernel<T, 1>)
                : (wide ? tree_merge_kernel<T, 2> : tree_merge_kernel<T, 1>);
  };
  return launch_behind(a.c.dtype == DSPARK_F32 ? pick(0.0f) : pick(__nv_bfloat16()), grid,
                       32 * kMergeWarps, 0, stream, a);
}

}  // namespace dspark
