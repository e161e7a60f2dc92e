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
// taken that their error could decide, those few are scored again in 64 bits.
// The error of a score is below eps = n 2^-24 A, A = the largest sum of |q_d| times
// the largest |bound|.  A product of the tensor cores adds 16 exact terms to a float32
// sum, off by at most 17 truncations of 2^-24 of what the terms may sum to; a score is
// kSums = 4 sums of D / 32 such products, added in float32: 17 D / 32 + 4 together, and
// n is twice that.  (One sum over all would have n = 4 D and send 25 lists of a hundred
// to be scored again, not 7.)  On the FFMA units a lane rounds D / 4 products and sums,
// and three more follow: n = D / 4 + 4.
//
// The scores are a pass over the bounds (2 D values a page and head against
// 2 D page_size of keys and values).  q+, q- and bounds of bfloat16 are bfloat16
// numbers: nothing is rounded but the sums.
#include <climits>
#include <cmath>

#include "dspark_common.cuh"
#include "host_util.cuh"
#include "select_pages.cuh"

namespace dspark {
namespace {

using namespace sm100;

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

constexpr uint32_t kSpin = 1u << 22;

// A wait, which mostly is over at its first poll: only then are others timed (all
// lanes of all warps reading the clock at each wait took a hundred times the work).
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, kSpin); }
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void copy16(void* to, uint64_t from, bool there) {
  const int n = there ? 16 : 0;  // else zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(n)
               : "memory");
}

// On the tensor cores: bfloat16, head_dim up to D = 64 or 128, filled up with zeros
// (heads of 96, 88 x 8 lists of 8 heads and up to 250 pages: 35 us, 88 with the FFMA form's scores).  An item is 128 pages of a
// sequence's key head, one row of 2 D bounds each; of the query rows up to N go with
// them at a time, q- and q+ behind one another: S [page][row] = (lo | hi) (q- | q+)^T into tensor memory, as kSums sums of
// D / 2 terms each.  A thread then has a page, takes the largest score of each token's
// heads and writes it beside its neighbours'.
//   warps 0..7    what comes of the scores, and the largest |bound| of each page:
//                 four warps an item, in turn
//   warps 8..11   bounds, two items ahead, a row of 256 or 512 bytes (two, one) at a
//                 time (copies by TMA, whose gather of four rows takes some 100 cycles,
//                 and bulk copies of one were three times slower)
//   warps 12..15  queries, two row tiles ahead, and their sums of |q|
//   warp 16       products
// One block a multiprocessor goes through the items of all sequences, in strides.
// (Blocks of one item each, with mma.sync or tcgen05, took 26 to 41 us for 7300 x 16
// pages where this takes 22: their loads were under way for a fifth of their time.)
constexpr int kSums = 4, kScorePages = 128, kScoreThreads = 544;
constexpr int kMaxB = DSPARK_CACHE_MAX_B;

struct Control {
  uint64_t a_full[2], a_empty[2], b_full[2], b_empty[2], t_empty[2];
  // scores are there, of each team: a wait is for a phase's parity, so nobody may wait
  // on a barrier some of whose phases it has passed over
  uint64_t t_full[2][2];
  uint64_t drain;   // all products are done
  uint32_t tmem;
  int failed;
  float sum_q[2][64];  // of a row tile's rows, and of the one with sums before it
  uint32_t named[2][4];  // the rows of both slots that are pages
  int warps[33];
  int offset[kMaxB + 1];  // items of the sequences before
  int seq[kMaxB], F[kMaxB];
  uint8_t tokens[kMaxB];
};

template <int D>
constexpr size_t score_tc_bytes(int N) {
  return 1024 + (size_t)2 * (kScorePages + N) * 4 * D + sizeof(Control);
}
static_assert(score_tc_bytes<128>(64) <= 232448, "shared memory of a block");

// A role's place in a pair of slots: the slot, and the parity of its phase.
struct Slot {
  int i;
  uint32_t parity;
  __device__ __forceinline__ void step() {
    i ^= 1;
    parity ^= i == 0;
  }
};

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(bar, parity));
}

struct Item {
  int b, h, page0, F, s, tokens;
};

template <int D>
__global__ void __launch_bounds__(kScoreThreads, 1)
    score_tc_kernel(const __grid_constant__ SelectArgs a, int N, int stall) {
  constexpr int kWords = D / 4;        // 16-byte words of a row of bounds, half as many of a query
  constexpr int kParts = 2 * D / 64;   // 128-byte parts of a row: the layout of the operands
  constexpr int kBytes = kScorePages * 4 * D;
  extern __shared__ uint8_t raw[];
  uint8_t* const A = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* const B = A + 2 * kBytes;
  Control& sh = *reinterpret_cast<Control*>(B + 2 * N * 4 * D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dim = a.c.head_dim;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.a_full[i], 4);
      mbar_init(&sh.a_empty[i], 5);
      mbar_init(&sh.b_full[i], 4);
      mbar_init(&sh.b_empty[i], 1);
      mbar_init(&sh.t_full[0][i], 1);
      mbar_init(&sh.t_full[1][i], 1);
      mbar_init(&sh.t_empty[i], 4);
    }
    mbar_init(&sh.drain, 1);
    sh.failed = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&sh.tmem, 2 * kSums * N);
    tmem_relinquish();
  }
  follow();
  for (int b = threadIdx.x; b < a.B; b += kScoreThreads) {
    const Seq q = find_seq(a, b, blockIdx.x == 0);
    sh.seq[b] = q.s;
    sh.F[b] = q.F;
    sh.tokens[b] = (uint8_t)q.tokens;
    sh.offset[b] = q.F > a.count && q.tokens > 0 ? (q.F + kScorePages - 1) / kScorePages * a.c.kv_heads : 0;
  }
  tc_fence_before();
  __syncthreads();
  row_offsets(sh.offset, sh.offset, a.B, sh.warps);  // synchronises the block
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int items = sh.offset[a.B], fit = N / a.group;  // tokens of a row tile
  // Item i, for a warp that asks for ever later ones.
  int b_now = 0;
  auto item = [&](int i) {
    while (true) {
      const int b = b_now + 1 + lane;
      const int n = __popc(__ballot_sync(0xffffffffu, b < a.B && sh.offset[b] <= i));
      b_now += n;
      if (n < 32) break;
    }
    Item x;
    x.b = b_now;
    x.F = sh.F[x.b];
    x.s = sh.seq[x.b];
    x.tokens = sh.tokens[x.b];
    const uint32_t tiles = (uint32_t)(x.F + kScorePages - 1) / kScorePages, at = (uint32_t)(i - sh.offset[x.b]);
    x.h = (int)(at / tiles);
    x.page0 = (int)(at - x.h * tiles) * kScorePages;
    return x;
  };
  bool ok = true;
  if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------------- bounds
    constexpr int kTogether = 32 / kWords;  // rows at a time
    const int part = lane / kWords, w = lane - part * kWords, row0 = (warp - 8) * 32;
    // the word of a row in memory, where dims may be fewer than D, or zeros
    const int side = w / (D / 8), word = side * (dim / 8) + w - side * (D / 8);
    const bool filled = w - side * (D / 8) < dim / 8;
    // where the rows of an item lie, one a lane (0: nowhere)
    auto rows_of = [&](int i) -> uint64_t {
      if (i >= items) return 0;
      const Item x = item(i);
      const int page = x.page0 + row0 + lane;
      if (page >= x.F) return 0;
      const int id = cache_page(a.c, x.s, page, a.c.max_pages);
      if (id < 0) {
        cache_error(a.c, kCacheErrPage);
        return 0;
      }
      return reinterpret_cast<uint64_t>(a.bounds) + bounds_row(a.c, a.layer, id, x.h);
    };
    Slot at{0, 1}, last{0, 0};  // the phase that frees a slot: the first round passes
    uint64_t next = rows_of(blockIdx.x);
    bool any = false;
    auto ready = [&]() {  // this warp's part of the item before is there
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.a_full[last.i]);
      last.step();
    };
#pragma unroll 1
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const uint64_t from = next;
      next = rows_of(i + gridDim.x);
      ok = wait_warp(&sh.a_empty[at.i], at.parity);
      if (!ok) break;
      const uint32_t there = __ballot_sync(0xffffffffu, from != 0);
      if (lane == 0) sh.named[at.i][warp - 8] = there;
      uint8_t* const to = A + at.i * kBytes + (w >> 3) * (kScorePages * 128) + (row0 + part) * 128;
#pragma unroll 4
      for (int r = 0; r < 32; r += kTogether) {
        const uint64_t row = __shfl_sync(0xffffffffu, from, r + part);
        const bool some = row != 0 && filled;
        copy16(to + r * 128 + (((w & 7) ^ ((r + part) & 7)) << 4),
               some ? row + 16 * word : reinterpret_cast<uint64_t>(a.bounds), some);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      at.step();
      if (any) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        ready();
      }
      any = true;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (any) ready();
  } else if (warp >= 12 && warp < 16) {
    // --------------------------------------------------------------- queries
    constexpr int kLanes = kWords / 2, kTogether = 32 / kLanes;  // lanes of a row, rows at a time
    constexpr int kStep = 4 * kTogether;                          // rows of four warps
    const int part = lane / kLanes, w = lane - part * kLanes, row0 = (warp - 12) * kTogether + part;
    Slot at{0, 1};
    int turn = 0;
    // failure-path test: one of them has given up
    if (stall == kStallAlone && warp == 13) ok = false;
#pragma unroll 1
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
      const Item x = item(i);
#pragma unroll 1
      for (int t0 = 0; t0 < x.tokens; t0 += fit) {
        const int tokens = x.tokens - t0 < fit ? x.tokens - t0 : fit, rows = tokens * a.group;
        const char* const from =
            a.q + (((size_t)x.b * a.T + t0) * a.heads + (size_t)x.h * a.group) * dim * 2 + 16 * w;
        uint8_t* const to = B + at.i * (N * 4 * D) + (w >> 3) * (N * 128);
        float* const sums = sh.sum_q[turn];
        uint4 q[4];
        auto load = [&](int r0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r0 + k * kStep + row0, t = r / a.group;
            q[k] = make_uint4(0, 0, 0, 0);
            if (r < rows && w < dim / 8)
              q[k] = *reinterpret_cast<const uint4*>(from + ((size_t)t * a.heads + (r - t * a.group)) * dim * 2);
          }
        };
        load(0);
        ok = wait_warp(&sh.b_empty[at.i], at.parity);
        if (!ok) break;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 4 * kStep) {
          if (r0 > 0) load(r0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r0 + k * kStep + row0;
            if (r < N) {  // behind the last row: zeros, or what was there
              uint8_t* row = to + r * 128 + (((w & 7) ^ (r & 7)) << 4);
              *reinterpret_cast<uint4*>(row) =
                  make_uint4(min_nan2(q[k].x, 0), min_nan2(q[k].y, 0), min_nan2(q[k].z, 0), min_nan2(q[k].w, 0));
              *reinterpret_cast<uint4*>(row + kParts / 2 * (N * 128)) =
                  make_uint4(max_nan2(q[k].x, 0), max_nan2(q[k].y, 0), max_nan2(q[k].z, 0), max_nan2(q[k].w, 0));
            }
            if (x.page0 == 0) {
              const uint32_t u[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
              float s = 0.0f;
#pragma unroll
              for (int n = 0; n < 4; ++n)
                s += fabsf(__uint_as_float(u[n] << 16)) + fabsf(__uint_as_float(u[n] & 0xffff0000u));
#pragma unroll
              for (int n = kLanes / 2; n > 0; n >>= 1) s += __shfl_xor_sync(0xffffffffu, s, n);
              if (w == 0 && r < rows) sums[r] = s;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.b_full[at.i]);
        if (x.page0 == 0) {  // the largest sum of each token's heads
          // the four warps' sums are there (and the other ones used up); a warp that has
          // given up does not come, and the wait for it runs out
          ok = wait_warp(&sh.b_full[at.i], at.parity ^ 1);
          turn ^= 1;
          if (!ok) break;
          for (int t = threadIdx.x - 12 * 32; t < tokens; t += 128) {
            float best = 0.0f;
            for (int g = 0; g < a.group; ++g) best = max_nan(best, sums[t * a.group + g]);
            a.reach_q[((size_t)x.b * a.T + t0 + t) * a.c.kv_heads + x.h] = best;
          }
          __syncwarp();
        }
        at.step();
      }
    }
  } else if (warp == 16) {
    // -------------------------------------------------------------- products
    const uint32_t idesc = idesc_bf16_f32(kScorePages, N, 0, 0);
    const uint64_t da0 = smem_desc_sw128(smem_u32(A), 16, 1024), db0 = smem_desc_sw128(smem_u32(B), 16, 1024);
    Slot as{0, 0}, bs{0, 0}, ts{0, 1};
    int turn = 0;  // the team that takes the item
#pragma unroll 1
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x, turn ^= 1) {
      const Item x = item(i);
      ok = wait_warp(&sh.a_full[as.i], as.parity);
      // failure-path test: bounds are there, and nothing completes this phase
      if (stall == kStallWait) ok = __all_sync(0xffffffffu, ok && mbar_wait(&sh.t_full[0][0], 0, kStallPolls));
#pragma unroll 1
      for (int t0 = 0; t0 < x.tokens && ok; t0 += fit) {
        ok = wait_warp(&sh.b_full[bs.i], bs.parity) && wait_warp(&sh.t_empty[ts.i], ts.parity);
        if (!ok) break;
        tc_fence_after();
        const uint64_t da = da0 + ((as.i * kBytes) >> 4), db = db0 + ((bs.i * (N * 4 * D)) >> 4);
        const uint32_t to = tmem + ts.i * kSums * N;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k) {
            constexpr int kEach = 2 * D / 16 / kSums;
            mma_bf16(to + (k / kEach) * N, da + (((k >> 2) * (kScorePages * 128) + (k & 3) * 32) >> 4),
                     db + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc, k % kEach != 0);
          }
          mma_commit(&sh.t_full[turn][ts.i]);
          mma_commit(&sh.b_empty[bs.i]);
          if (t0 + fit >= x.tokens) mma_commit(&sh.a_empty[as.i]);
        }
        __syncwarp();
        bs.step();
        ts.step();
      }
      as.step();
    }
    // tensor memory is given back behind the last of them
    if (elect_one()) mma_commit(&sh.drain);
    wait_warp(&sh.drain, 0);
  } else {
    // ---------------------------------------------------------------- scores
    Slot as{0, 0};
    int slot = 0;         // of the next tile's scores
    uint32_t phases = 0;  // bit i: the parity of this team's next phase in slot i
    const int team = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const bool together = a.lists == 1;
    const size_t list_step = (size_t)a.c.kv_heads * a.stride;
    int turn = 0;
#pragma unroll 1
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x, turn ^= 1) {
      const Item x = item(i);
      if (turn != team) {  // the other four warps'
        as.step();
        for (int t0 = 0; t0 < x.tokens; t0 += fit) slot ^= 1;
        continue;
      }
      const int page = x.page0 + row;
      float* at = a.scores + list_row(a, x.b, 0, x.h) * a.stride + page;
      ok = wait_warp(&sh.a_full[as.i], as.parity);
      if (!ok) break;
      const bool there = page < x.F, named = (sh.named[as.i][quarter] >> lane) & 1;
      {  // the largest |bound| of the thread's page, and of its neighbours
        uint32_t low = 0, high = 0;
        const uint8_t* const from = A + as.i * kBytes + row * 128;
#pragma unroll 8
        for (int w = 0; w < kWords; ++w) {
          const uint4 u = *reinterpret_cast<const uint4*>(from + (w >> 3) * (kScorePages * 128) +
                                                          (((w & 7) ^ (row & 7)) << 4));
          low = min_nan2(min_nan2(low, u.x), min_nan2(min_nan2(u.y, u.z), u.w));
          high = max_nan2(max_nan2(high, u.x), max_nan2(max_nan2(u.y, u.z), u.w));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.a_empty[as.i]);
        uint32_t m = max_nan2(low ^ 0x80008000u, high);
        m = max_nan2(m, m >> 16 | m << 16);
#pragma unroll
        for (int k = kReachPages / 2; k > 0; k >>= 1) m = max_nan2(m, __shfl_xor_sync(0xffffffffu, m, k));
        if ((lane & (kReachPages - 1)) == 0 && there)
          a.reach_k[((size_t)x.b * a.c.kv_heads + x.h) * a.reaches + page / kReachPages] = __uint_as_float(m << 16);
      }
      as.step();
      float run = -INFINITY;
#pragma unroll 1
      for (int t0 = 0; t0 < x.tokens; t0 += fit) {
        const int tokens = x.tokens - t0 < fit ? x.tokens - t0 : fit, rows = tokens * a.group;
        ok = wait_warp(&sh.t_full[team][slot], (phases >> slot) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = tmem + slot * kSums * N + ((uint32_t)(quarter * 32) << 16);
        float best = -INFINITY;
        int left = a.group;  // rows of the token
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8) {
          uint32_t v[kSums][8];
#pragma unroll
          for (int k = 0; k < kSums; ++k) tmem_ld8(from + k * N + r0, v[k]);
          tmem_ld_wait();
          const int n_rows = rows - r0;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float s = (__uint_as_float(v[0][n]) + __uint_as_float(v[1][n])) +
                            (__uint_as_float(v[2][n]) + __uint_as_float(v[3][n]));
            if (n < n_rows) {
              best = fmaxf(best, kept(s));
              if (--left == 0) {
                if (!named) best = -INFINITY;
                if (together) {
                  run = fmaxf(run, best);
                } else {
                  if (there) *at = best;
                  at += list_step;
                }
                best = -INFINITY;
                left = a.group;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.t_empty[slot]);
        phases ^= 1u << slot;
        slot ^= 1;
      }
      if (together && there) *at = run;
    }
  }
  if (!ok) sh.failed = 1;
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kSums * N);
  }
  if (threadIdx.x == 0 && sh.failed) cache_error(a.c, kDevErrTimeout);
}

// On the FFMA units: a warp takes 8 pages, four lanes each, and eight query rows at a
// time, of 32 that the block holds.  Bounds and queries are staged in shared memory, a
// bulk copy for each row, which a lane issues (16 bytes a lane and copy took 450
// cycles a page to issue).
constexpr int kScoreWarps = 4, kScoreRows = 32;

// Bytes from one row in shared memory to the next: an odd multiple of 64, so that
// what eight lanes read of two rows lies in different banks.
__host__ __device__ __forceinline__ int pitch_of(int bytes) { return (bytes + 63) / 64 / 2 * 128 + 64; }

template <typename T>
int score_ffma_bytes(int D) {
  return kScoreWarps * kReachPages * pitch_of(2 * D * (int)sizeof(T)) + kScoreRows * pitch_of(D * (int)sizeof(T));
}

// s + max(q lo, q hi) for finite numbers; where the bounds or q are not, every
// page is scored in 64 bits.
__device__ __forceinline__ float reach(float q, float lo, float hi, float s) {
  return fmaf(q, q < 0.0f ? lo : hi, s);
}

template <typename T>
__global__ void __launch_bounds__(32 * kScoreWarps) score_ffma_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kTake = 8, kPages = kReachPages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t ready[kScoreWarps + 1];  // a warp's bounds; the queries
  follow();
  const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3, D = a.c.head_dim;
  const int bound_bytes = 2 * D * (int)sizeof(T), query_bytes = D * (int)sizeof(T);
  const int bound_pitch = pitch_of(bound_bytes), query_pitch = pitch_of(query_bytes);
  uint8_t* const bounds = smem + warp * kPages * bound_pitch;
  uint8_t* const queries = smem + kScoreWarps * kPages * bound_pitch;
  const Seq seq = find_seq(a, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  const int first = blockIdx.x * kScoreWarps * kPages, all = gridDim.x * kScoreWarps * kPages;
  if (seq.F <= a.count || seq.tokens == 0 || first >= seq.F) return;
  const int fit = kScoreRows / a.group;  // tokens of a tile
  const bool together = a.lists == 1;
  float* const scores = a.scores + list_row(a, b, 0, h) * a.stride;
  const size_t list_step = (size_t)a.c.kv_heads * a.stride;
  if (threadIdx.x <= kScoreWarps) mbar_init(&ready[threadIdx.x], 1);
  fence_mbar_init();
  __syncthreads();
  uint32_t bound_phase = 0, query_phase = 0;
  bool ok = true;
#pragma unroll 1
  for (int block0 = first; block0 < seq.F; block0 += all) {
    const int page0 = block0 + warp * kPages, page = page0 + gid;
    const int id = page < seq.F ? cache_page(a.c, seq.s, page, a.c.max_pages) : -1;
    if (page < seq.F && id < 0) cache_error(a.c, kCacheErrPage);
    if (page0 < seq.F) {
      const uint32_t there = __ballot_sync(0xffffffffu, tig == 0 && id >= 0);
      if (lane == 0) mbar_arrive_expect_tx(&ready[warp], __popc(there) * bound_bytes);
      __syncwarp();
      if (tig == 0 && id >= 0)
        copy_bulk(bounds + gid * bound_pitch, a.bounds + bounds_row(a.c, a.layer, id, h), bound_bytes, &ready[warp]);
    }
    float reach_k = 0.0f, run = -INFINITY;
#pragma unroll 1
    for (int t0 = 0; t0 < seq.tokens; t0 += fit) {
      const int tokens = seq.tokens - t0 < fit ? seq.tokens - t0 : fit, rows = tokens * a.group;
      if (t0 > 0) {  // the tile before is used up, and copied over
        fence_proxy_async_smem();
        __syncthreads();
      }
      if (t0 > 0 || block0 == first || seq.tokens > fit) {
        if (warp == 0) {
          if (lane == 0) mbar_arrive_expect_tx(&ready[kScoreWarps], rows * query_bytes);
          __syncwarp();
          const int t = lane / a.group;
          if (lane < rows)
            copy_bulk(queries + lane * query_pitch,
                      a.q + (((size_t)b * a.T + t0 + t) * a.heads + (size_t)h * a.group + (lane - t * a.group)) * query_bytes,
                      query_bytes, &ready[kScoreWarps]);
        }
        ok = wait(&ready[kScoreWarps], query_phase) && ok;
        query_phase ^= 1;
      }
      if (t0 == 0 && page0 < seq.F) {
        ok = wait(&ready[warp], bound_phase) && ok;
        bound_phase ^= 1;
      }
      if (blockIdx.x == 0 && block0 == 0) {
        // the largest sum of |q| of each token's heads
        for (int t = warp; t < tokens; t += kScoreWarps) {
          float best = 0.0f;
          for (int g = 0; g < a.group; ++g) {
            const T* q = reinterpret_cast<const T*>(queries + (t * a.group + g) * query_pitch);
            float x = 0.0f;
            for (int d = 4 * lane; d < D; d += 128) {
              const float4 v = load4<T>(q + d);
              x += fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w);
            }
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
            best = max_nan(best, x);
          }
          if (lane == 0) a.reach_q[((size_t)b * a.T + t0 + t) * a.c.kv_heads + h] = best;
        }
      }
      if (page0 >= seq.F) continue;
      const T* lo = reinterpret_cast<const T*>(bounds + gid * bound_pitch);
      float best = -INFINITY;
      int g = 0, t = 0;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += kTake) {
        float s[kTake];
#pragma unroll
        for (int i = 0; i < kTake; ++i) s[i] = 0.0f;
#pragma unroll 2
        for (int d = 4 * tig; d < D; d += 16) {
          const float4 l = load4<T>(lo + d), u = load4<T>(lo + D + d);
          if (t0 == 0 && r0 == 0 && id >= 0) {
            reach_k = max_nan(reach_k, max_nan(max_nan(fabsf(l.x), fabsf(l.y)), max_nan(fabsf(l.z), fabsf(l.w))));
            reach_k = max_nan(reach_k, max_nan(max_nan(fabsf(u.x), fabsf(u.y)), max_nan(fabsf(u.z), fabsf(u.w))));
          }
#pragma unroll
          for (int i = 0; i < kTake; ++i) {  // rows behind the last: whatever lies there
            const float4 x = load4<T>(reinterpret_cast<const T*>(queries + (r0 + i) * query_pitch) + d);
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
            if (id < 0) best = -INFINITY;
            if (together) run = fmaxf(run, best);
            else if (tig == 0 && page < seq.F) scores[(t0 + t) * list_step + page] = best;
            best = -INFINITY;
            g = 0;
            ++t;
          }
        }
      }
    }
    if (page0 < seq.F) {
      if (together && tig == 0 && page < seq.F) scores[page] = run;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) reach_k = max_nan(reach_k, __shfl_xor_sync(0xffffffffu, reach_k, x));
      if (lane == 0) a.reach_k[((size_t)b * a.c.kv_heads + h) * a.reaches + page0 / kReachPages] = reach_k;
    }
    if (block0 + all < seq.F) {  // queries and bounds are used up, and copied over
      fence_proxy_async_smem();
      __syncthreads();
    }
  }
  if (!ok) cache_error(a.c, kDevErrTimeout);
}

// --------------------------------------------------------------- selection
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
    int count[W > 1 ? 8 * W : 1];  // of stretches and warps
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
  // Places before this thread among those whose flag is set; adds all to `n`.
  __device__ __forceinline__ int place(bool flag, int& n) {
    const int lane = thread & 31, warp = thread >> 5;
    const uint32_t m = __ballot_sync(0xffffffffu, flag);
    int at = n + __popc(m & ((1u << lane) - 1));
    if (W == 1) {
      n += __popc(m);
      return at;
    }
    if (lane == 0) sh.part[turn][warp] = __popc(m);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int k = (int)sh.part[turn][i];
      if (i < warp) at += k;
      n += k;
    }
    turn ^= 1;
    return at;
  }
};

// q times the bound that makes the larger product, exact.
__device__ __forceinline__ double larger(float q, float lo, float hi) {
  return (double)q * (q < 0.0f ? lo : hi);
}
// A sum of terms x, |x| < 2^22 together, in three float32 numbers: multiples of 1, of
// 2^-16 and of 2^-32, what is left of a term going from one to the next.  Up to 256
// terms (and as many remainders of products) leave each below 2^24 of its multiples,
// so the sums are exact, and off by 2^-33 a term in all.
struct Exact {
  float n[3] = {0.0f, 0.0f, 0.0f};
  template <int kFrom>
  __device__ __forceinline__ void add(float x) {
    constexpr float magic[3] = {0x1.8p23f, 0x1.8p7f, 0x1.8p-9f};  // rounds to a multiple
#pragma unroll
    for (int i = kFrom; i < 3; ++i) {
      const float m = __fsub_rn(__fadd_rn(x, magic[i]), magic[i]);
      n[i] += m;
      x -= m;
    }
  }
  // in multiples of 2^-32
  __device__ __forceinline__ long long value() const {
    return ((long long)(int)n[0] << 32) + ((long long)(int)(n[1] * 0x1p16f) << 16) + (int)(n[2] * 0x1p32f);
  }
};
// Adds q times the bound that makes the larger product: of bfloat16 numbers it is
// exact in float32, of float32 numbers with the remainder that a fused product gives.
template <typename T>
__device__ __forceinline__ void add_larger(Exact& s, float q, float lo, float hi, float scale) {
  const float x = q < 0.0f ? lo : hi, p = q * x;
  s.add<0>(p * scale);
  if (sizeof(T) == 4) s.add<1>(fmaf(q, x, -p) * scale);
}

// What a list goes by: `tokens` tokens from t0 on of a sequence's key head.
struct List {
  int b, h, t0, tokens;
  Seq seq;
};

// Scores of four pages in 64 bits, eight lanes each (page -1: there is none), as bits
// whose order is theirs: of scale times the products in float32 numbers whose sums are
// exact, or where scale is 0 (infinities, extreme sizes) in double.  (The 64-bit
// floating-point units, which convert to 64-bit integers too, have a sixty-fourth of
// the others' rate: with them the selection of 5632 lists took 67 us of 97.)
template <typename T>
__device__ __noinline__ uint64_t exact_scores(const SelectArgs& a, const List& l, int page, float scale, int lane) {
  const int D = a.c.head_dim, id = page < 0 ? -1 : cache_page(a.c, l.seq.s, page, a.c.max_pages);
  const int first = 4 * (lane & 7);
  const T* lo = reinterpret_cast<const T*>(a.bounds + bounds_row(a.c, a.layer, id < 0 ? 0 : id, l.h)) + first;
  const size_t token = (size_t)a.heads * D;
  const T* q = reinterpret_cast<const T*>(a.q) +
               ((size_t)l.b * a.T + l.t0) * token + (size_t)l.h * a.group * D + first;
  const int rows = l.tokens * a.group;
  long long most = LLONG_MIN;
  double best = -INFINITY;
  int g = 0;  // the head of the next row
  if (scale > 0.0f) {
    // rows whose loads are in flight together (4: 38.4 us for the 5632 lists, 2: 35.6,
    // whose registers the kernel's other parts would have to give up, 1: 37.0)
    constexpr int kTake = 2;
#pragma unroll 1
    for (int r = 0; r < rows; r += kTake) {
      const T* at[kTake];
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        at[i] = q;  // the last row again where there are no more
        if (r + i + 1 < rows) {
          q += D;
          if (++g == a.group) {
            g = 0;
            q += token - (size_t)a.group * D;
          }
        }
      }
      Exact s[kTake];
#pragma unroll 2
      for (int d = 0; d < D - first; d += 32) {
        const float4 y = load4<T>(lo + d), z = load4<T>(lo + D + d);
        float4 x[kTake];
#pragma unroll
        for (int i = 0; i < kTake; ++i) x[i] = load4<T>(at[i] + d);
#pragma unroll
        for (int i = 0; i < kTake; ++i) {
          add_larger<T>(s[i], x[i].x, y.x, z.x, scale);
          add_larger<T>(s[i], x[i].y, y.y, z.y, scale);
          add_larger<T>(s[i], x[i].z, y.z, z.z, scale);
          add_larger<T>(s[i], x[i].w, y.w, z.w, scale);
        }
      }
#pragma unroll
      for (int k = 4; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < kTake; ++i)
#pragma unroll
          for (int n = 0; n < 3; ++n) s[i].n[n] += __shfl_xor_sync(0xffffffffu, s[i].n[n], k);
#pragma unroll
      for (int i = 0; i < kTake; ++i) {
        const long long v = s[i].value();
        most = v > most ? v : most;
      }
    }
  } else {
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
      double s = 0.0;
#pragma unroll 1
      for (int d = 0; d < D - first; d += 32) {
        const float4 x = load4<T>(q + d), y = load4<T>(lo + d), z = load4<T>(lo + D + d);
        s += larger(x.x, y.x, z.x) + larger(x.y, y.y, z.y) + larger(x.z, y.z, z.z) + larger(x.w, y.w, z.w);
      }
#pragma unroll
      for (int i = 4; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
      best = s == s ? fmax(best, s) : INFINITY;
      q += D;
      if (++g == a.group) {
        g = 0;
        q += token - (size_t)a.group * D;
      }
    }
  }
  if (id < 0) return 0;
  return scale > 0.0f ? (uint64_t)most ^ (1ull << 63) : ordered_bits64(best);
}

// Writes one list: `scores` of the sequence's F > count pages, sums of terms whose
// sizes add up to size_of() at most (0 only where all scores are); border: room for F numbers.  A
// thread holds the first R of its scores as bits whose order is theirs (read anew from
// memory and made each time they took a third of the time).
template <typename T, int W, int R, typename Size>
__device__ __forceinline__ void pick_list(const SelectArgs& a, const List& l, const float* scores, Size size_of,
                                          uint64_t* border, Team<W>& team, int32_t* out) {
  constexpr int kSize = 32 * W;
  const int tid = team.thread, lane = tid & 31, F = l.seq.F;
  const int lo = a.first, hi = F - a.last, want = a.count - a.first - a.last;
  // 0 (below every score's) where there is no candidate; -0 is 0
  auto key_of = [&](int j) { return j >= lo && j < hi ? ordered_bits(scores[j] + 0.0f) : 0u; };
  uint32_t held[R];
#pragma unroll
  for (int i = 0; i < R; ++i) held[i] = key_of(i * kSize + tid);
  const float size = size_of();
  // f(page, key) of all that are this thread's
  auto all = [&](auto f) {
#pragma unroll
    for (int i = 0; i < R; ++i) f(i * kSize + tid, held[i]);
#pragma unroll 1
    for (int j = R * kSize + tid; j < F; j += kSize) f(j, key_of(j));
  };
  // What decides: pages with keys from `edge` on are taken, and of the `listed`
  // others from `near` on those that the exact scores say: the list in shared memory
  // names the taken ones, or, of many, the ones above `cut` are taken and the first
  // `ties` that equal it.
  uint32_t edge = ~0u, near = ~0u;
  bool many = false;
  int listed = 0, ties = 0;
  uint64_t cut = ~0ull;
  if (want > 0) {
    uint32_t least = ~0u, most = 0;
    all([&](int, uint32_t k) {
      least = k && k < least ? k : least;
      most = k > most ? k : most;
    });
    // `want` keys are at or above `at`, or more, and then all below at + 1
    uint32_t at = team.least(least), above = team.most(most) + 1;
    bool split = false;
#pragma unroll 1
    while (!split && above - at > 1) {
      const uint32_t mid = at + (above - at) / 2;
      uint32_t n = 0;
      all([&](int, uint32_t k) { n += k >= mid; });
      n = team.sum(n);
      split = n == (uint32_t)want;
      if (n >= (uint32_t)want) at = mid;
      else above = mid;
    }
    uint32_t in = ~0u, below = 0;  // the lowest that is taken, the highest that is not
    all([&](int, uint32_t k) {
      if (k >= at) in = k < in ? k : in;
      else below = k > below ? k : below;
    });
    edge = team.least(in);
    below = split ? team.most(below) : edge;
    const float last = from_ordered_bits(edge);
    const float eps = a.error * size;
    // eps grows with the terms, and below 2^-126 float32 rounds by a fixed step, or
    // drops a term whole: of sums that small nothing is known
    const bool small = size > 0.0f && size < 0x1p-90f;
    if (small || !(last - from_ordered_bits(below) > 2.0f * eps)) {
      // scores within 2 eps of the last one that is taken could change places
      const bool known = !small && size <= 0x1p100f && fabsf(last) <= 0x1p101f;
      // sums below 2^22; a product that float32 cannot hold whole is far below 2^-32
      const float scale = size == 0.0f ? 1.0f
                          : known && size >= 0x1p-60f ? __int_as_float((127 + 21 - ilogbf(size)) << 23) : 0.0f;
      near = known ? ordered_bits(last - 2.0f * eps) : 1u;
      edge = known ? ordered_bits(last + 2.0f * eps) + 1 : ~0u;
      if (tid == 0) team.sh.n = 0;
      team.sync();
      uint32_t sure = 0, m = 0;
      all([&](int j, uint32_t k) {
        sure += k >= edge;
        if (k >= near && k < edge) {
          ++m;
          const int i = atomicAdd(&team.sh.n, 1);
          if (i < kNear) team.sh.near[i] = j;
        }
      });
      const int need = want - (int)team.sum(sure);
      listed = (int)team.sum(m);
      many = listed > kNear;
      if (listed == need) {  // all of them
        edge = near;
        many = false;
        listed = 0;
      } else if (!many) {
        team.sync();
#pragma unroll 1
        for (int e0 = 4 * (tid >> 5); e0 < listed; e0 += 4 * W) {
          const int e = e0 + (lane >> 3);
          const uint64_t x = exact_scores<T>(a, l, e < listed ? team.sh.near[e] : -1, scale, lane);
          if (e < listed && (lane & 7) == 0) team.sh.exact[e] = x;
        }
        team.sync();
        // rank by score, then by place; those that stay out are struck off
        bool out_of = false;
        if (tid < listed) {
          const uint64_t x = team.sh.exact[tid];
          const int j = team.sh.near[tid];
          int rank = 0;
          for (int e = 0; e < listed; ++e) {
            const uint64_t y = team.sh.exact[e];
            rank += y > x || (y == x && team.sh.near[e] < j);
          }
          out_of = rank >= need;
        }
        team.sync();
        if (out_of) team.sh.near[tid] = -1;
        team.sync();
      } else {
#pragma unroll 1
        for (int j0 = 0; j0 < F; j0 += kSize) {
          const int j = j0 + tid;
          const uint32_t k = key_of(j);
          uint32_t here = __ballot_sync(0xffffffffu, k >= near && k < edge);
          while (here) {
            uint32_t left = here;  // the next four
            for (int i = 0; i < lane >> 3; ++i) left &= left - 1;
            const int page = left ? j0 + (tid & ~31) + __ffs(left) - 1 : -1;
            const uint64_t x = exact_scores<T>(a, l, page, scale, lane);
            if (page >= 0 && (lane & 7) == 0) border[page] = x;
            for (int i = 0; i < 4; ++i) here &= here - 1;
          }
        }
        team.sync();
        // the need-th largest of them
        uint64_t low = 0, high = ~0ull;
#pragma unroll 1
        while (high - low > 1) {
          const uint64_t mid = low + (high - low) / 2;
          uint32_t n = 0;
#pragma unroll 1
          for (int j = tid; j < F; j += kSize) {
            const uint32_t k = key_of(j);
            n += k >= near && k < edge && border[j] >= mid;
          }
          n = team.sum(n);
          if (n >= (uint32_t)need) low = mid;
          else high = mid;
        }
        cut = low;
        uint32_t n = 0;
#pragma unroll 1
        for (int j = tid; j < F; j += kSize) {
          const uint32_t k = key_of(j);
          n += k >= near && k < edge && border[j] > cut;
        }
        ties = need - (int)team.sum(n);
      }
    }
  }
  // the taken pages in order
  int done = 0, tied = 0;
  auto write = [&](int j, uint32_t k) {
    bool take = j < lo || (j >= hi && j < F) || k >= edge;
    if (listed > 0) {
      const bool border_line = k >= near && k < edge;
      if (many) {  // of those on the border the first ones, as many as there is room for
        bool tie = false;
        if (border_line) {
          take = border[j] > cut;
          tie = border[j] == cut;
        }
        const int before = team.place(tie, tied);
        if (tie) take = before < ties;
      } else if (border_line) {
        for (int e = 0; e < listed; ++e) take |= team.sh.near[e] == j;
      }
    }
    const int at = team.place(take, done);
    if (take && at < a.count) out[at] = j;
  };
  if (many || F > R * kSize) {
#pragma unroll 1
    for (int j0 = 0; j0 < F; j0 += kSize) write(j0 + tid, key_of(j0 + tid));
    return;
  }
  // the counts of all stretches in one exchange
  uint32_t took[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int j = i * kSize + tid;
    bool take = j < lo || (j >= hi && j < F) || held[i] >= edge;
    if (listed > 0 && held[i] >= near && held[i] < edge)
      for (int e = 0; e < listed; ++e) take |= team.sh.near[e] == j;
    took[i] = __ballot_sync(0xffffffffu, take);
    if (W > 1 && lane == 0) team.sh.count[i * W + (tid >> 5)] = __popc(took[i]);
  }
  if (W > 1) team.sync();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i * kSize >= F) break;
    int at = 0;
    if (W > 1) {  // a lane: the takers of some stretches and warps, of those before this warp's
#pragma unroll
      for (int x = 0; x < R * W; x += 32)
        if (x + lane < i * W + (tid >> 5)) at += team.sh.count[x + lane];
      at = __reduce_add_sync(0xffffffffu, at);
    } else {
      at = done;
      done += __popc(took[i]);
    }
    at += __popc(took[i] & ((1u << lane) - 1));
    if ((took[i] >> lane) & 1 && at < a.count) out[at] = i * kSize + tid;
  }
}

// The largest of n numbers times the largest of m, by a warp; NaN if one is, and 0 only
// if all n or all m are.  All loads are under way before the first is used.
__device__ __forceinline__ float largest_product(const float* x, int n, size_t step_x, const float* y, int m,
                                                 int lane) {
  float u = 0.0f, v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = lane + 32 * k < m ? y[lane + 32 * k] : 0.0f;
  for (int i = lane; i < n; i += 32) u = max_nan(u, x[i * step_x]);
#pragma unroll 1
  for (int i = lane + 256; i < m; i += 32) v[0] = max_nan(v[0], y[i]);
#pragma unroll
  for (int k = 1; k < 8; ++k) v[0] = max_nan(v[0], v[k]);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    u = max_nan(u, __shfl_xor_sync(0xffffffffu, u, i));
    v[0] = max_nan(v[0], __shfl_xor_sync(0xffffffffu, v[0], i));
  }
  const float size = u * v[0];
  return size < 0x1p-126f && u > 0.0f && v[0] > 0.0f ? 0x1p-126f : size;
}

// ----------------------------------------------------------------- kernels
// Two launches: warps score stretches of pages, and one warp or eight pick a list.
// (One launch, in which a block scored a key head's pages into shared memory and picked
// its lists there, left multiprocessors idle behind the longest sequences: 42 us for
// 88 x 8 lists of 8 heads and up to 250 pages.)
constexpr int kPickWarps = 8;

template <typename T, int W, int R>
__global__ void __launch_bounds__(32 * kPickWarps, W == 1 && R == 8 ? 3 : 2)
    pick_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ typename Team<W>::Shared shared[kPickWarps / W];
  follow();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = W == 1 ? blockIdx.x * kPickWarps + warp : blockIdx.x;
  if (row >= a.B * a.lists * a.c.kv_heads) return;
  const int bt = row / a.c.kv_heads, h = row - bt * a.c.kv_heads;
  const int b = bt / a.lists, t = bt - b * a.lists;
  const Seq seq = find_seq(a, b, false);
  if (seq.F < 0 || t >= seq.tokens) return;
  Team<W> team(shared[W == 1 ? warp : 0], W == 1 ? lane : threadIdx.x);
  int32_t* out = a.pages + (size_t)row * a.count;
  if (seq.F <= a.count) {  // all pages
    for (int i = team.thread; i < a.count; i += 32 * W) out[i] = i < seq.F ? i : -1;
    return;
  }
  const List l{b, h, a.lists == 1 ? 0 : t, a.lists == 1 ? seq.tokens : 1, seq};
  pick_list<T, W, R>(
      a, l, a.scores + (size_t)row * a.stride,
      [&]() {
        return largest_product(a.reach_q + ((size_t)b * a.T + l.t0) * a.c.kv_heads + h, l.tokens, a.c.kv_heads,
                               a.reach_k + ((size_t)b * a.c.kv_heads + h) * a.reaches,
                               (seq.F + kReachPages - 1) / kReachPages, lane);
      },
      a.border + (size_t)row * a.stride, team, out);
}

template <typename T>
cudaError_t launch_pick(const SelectArgs& a, int sms, cudaStream_t stream) {
  // a warp for a list where lists are many and short enough for its registers
  const int rows = a.B * a.c.kv_heads * a.lists, size = 32 * kPickWarps;
  if (rows >= 4 * sms && a.c.max_pages <= 1024)
    return launch_behind(a.c.max_pages <= 256 ? pick_kernel<T, 1, 8> : pick_kernel<T, 1, 32>,
                         (rows + kPickWarps - 1) / kPickWarps, size, 0, stream, a);
  return launch_behind(pick_kernel<T, kPickWarps, 8>, rows, size, 0, stream, a);
}

// As many blocks as the table has stretches of `pages` for, unless the batch alone
// fills the GPU many times over; the blocks of short sequences end at once.
dim3 score_grid(const SelectArgs& a, int pages, int sms) {
  const int heads = a.B * a.c.kv_heads, most = (32 * sms + heads - 1) / heads;
  const int stretches = (a.c.max_pages + pages - 1) / pages;
  return dim3(stretches < most ? stretches : most, a.c.kv_heads, a.B);
}

template <int D>
cudaError_t launch_score_tc(const SelectArgs& a, int sms, cudaStream_t stream) {
  const int rows = a.T * a.group, N = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  // the limit is the kernel's, of all sizes: another thread may set it before the launch
  const cudaError_t e = cudaFuncSetAttribute(score_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)score_tc_bytes<D>(64));
  if (e != cudaSuccess) return e;
  return launch_behind(score_tc_kernel<D>, sms, kScoreThreads, score_tc_bytes<D>(N), stream, a, N,
                       stall_requested());
}

template <typename T>
cudaError_t launch_score_ffma(const SelectArgs& a, int sms, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(score_ffma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             score_ffma_bytes<T>(256));  // likewise
  if (e != cudaSuccess) return e;
  return launch_behind(score_ffma_kernel<T>, score_grid(a, kScoreWarps * kReachPages, sms), 32 * kScoreWarps,
                       score_ffma_bytes<T>(a.c.head_dim), stream, a);
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& args, int sms, cudaStream_t stream) {
  SelectArgs a = args;
  const int D = a.c.head_dim;
  const bool bf16 = a.c.dtype == DSPARK_BF16;
  const bool tc = bf16 && D <= 128;
  const int terms = D <= 64 ? 64 : 128;
  a.error = (tc ? 2 * (17 * (terms / 8 / kSums) + kSums) : D / 4 + 4) * 0x1p-24f;
  const cudaError_t e = tc      ? (D <= 64 ? launch_score_tc<64>(a, sms, stream) : launch_score_tc<128>(a, sms, stream))
                        : bf16 ? launch_score_ffma<__nv_bfloat16>(a, sms, stream)
                               : launch_score_ffma<float>(a, sms, stream);
  if (e != cudaSuccess) return e;
  return bf16 ? launch_pick<__nv_bfloat16>(a, sms, stream) : launch_pick<float>(a, sms, stream);
}

}  // namespace dspark
