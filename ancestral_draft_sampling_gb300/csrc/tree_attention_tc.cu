// tree_attention_tc.cu -- attention of drafted tokens over the paged cache on
// the 5th-generation tensor cores (tcgen05), bfloat16, head_dim 64 or 128.
//
// For 128 rows (drafted tokens times query heads) and each tile of 128 keys:
// S = Q K^T into tensor memory, weights P = 2^(c S - m) (c = scale log2 e)
// from one thread for each row back into tensor memory over S, O += P V.  m is
// the row's reference: the running maximum, but raised only when a tile's
// maximum passes it by more than 8 (weights stay below 2^8, sums far inside
// float32; any reference near the maximum gives the same quotient, and raising
// it seldom is a published method for attention on this chip), so O, which
// lives in tensor memory for the whole unit, is seldom rescaled.
//
// The sum l is taken of the float32 weights; the product reads them rounded to
// bfloat16 (at most 2^-8 of each, independent from key to key), which is what
// the tensor cores multiply beside bfloat16 values.  That is the one rounding to
// fewer bits, and it is a choice for speed: against 64 bits the root mean square
// error of the result relative to its own is 2.1e-3 to 2.3e-3 for one request,
// single tokens and wide trees (1.2e-3 for the full batch) where the rounding of
// the output alone makes 1.7e-3 (1.1e-3).  Weights split into two bfloat16
// numbers, both multiplied, have that error of 1.7e-3 (1.1e-3) and take a second
// set of products: single tokens 75.9 -> 86.1 us, full batch 534 -> 551 to 592, wide
// tree 69.5 -> 79.2 a replay.  The FFMA kernel multiplies float32 weights.
//
// Two streams share a block, each with S, O and four softmax warps of its own,
// so one stream's softmax runs under the other's products.  A unit of more
// than 128 rows gives each stream half the rows, and both use every tile of
// keys and values; a smaller unit gives each stream every other tile, and the
// two results are joined at its end.
//
// Narrow units, of at most 32 rows (T * group <= 32: single tokens, short
// chains), would leave three of a stream's four warps without rows.  Their
// queries are loaded four times, one below the other, so that every warp finds
// all the rows in its lanes and weighs a quarter of the tile's keys.  The
// weights go to shared memory (the product takes 128 rows from there, of which
// 32 count), the warps agree on m through shared memory where one of them
// raises it, and add up l at the unit's end (88 contexts of 600 keys 51.6 ->
// 49.2 us).
//
// Bound by HBM while rows * 4 flops for each key element stay below the
// tensor cores' rate, that is up to about 285 rows a key head; the layout
// follows from that: one block a multiprocessor, keys and values in rings of
// 32 KB (16 KB) tiles that TMA fills straight from the pages, 160 KB or more
// in flight, which covers the latency of HBM several times over.  Replays on
// one GB300, 8 key heads: 88 x 8 tokens over up to 16000 keys of 128 dims 534
// us, 6.8 TB/s, the rate of a copy; 44 single tokens with a window of 4096 keys
// of 64 dims 76 us, 4.5 TB/s: 1400 cycles a tile, which the chain scores -
// softmax - sums of each stream and the product warp bound alike (the same with
// the keys in L2; two product warps, both streams at once and waits handed to
// the softmax warps were no faster), and 8000 at each of a block's two or three
// unit ends; 8 trees of 61 tokens, 64 query heads, 5000 keys 69 us, 770 TFLOP/s,
// bound by the same chain: a pair of tiles takes 3470 cycles, of which the
// products take 2100.
//   warps 0, 3   fill the rings of keys and of values, a copy for each page's
//                rows and each half of the head (64 values, 128-byte swizzle);
//                the page numbers come 32 at a time, one load ahead.  Warp 3
//                also loads a unit's queries (rows (token, head) of the key
//                head), once the last unit's scores are done.
//   warp 1       issues the products.
//   warp 2       walks the block's units and describes them to the others, up
//                to four ahead (walks of their own made each role's code 8 KB
//                longer, and code comes from memory: 160 KB in all, of which a
//                unit of a few tiles waited for 9 us); tells the merge what to
//                do.
//   warps 4..7, 8..11  the streams' softmax: rows 32 (w % 4) .. + 31, or keys
//                32 (w % 4) .. + 31 of all rows of a narrow unit.
// Tiles that some rows see and others do not (the drafted tokens, a window's
// edge, the sequence's end) may hold NaN or infinities in places that weigh
// nothing, and 0 * NaN would reach every row.  Their values are looked
// through first; entries that are not finite are added to the rows that see
// them by hand and cleared.
//
// Every wait is bounded; where one runs out the kernel sets the error word,
// waits (bounded) for its copies and products, frees its tensor memory and
// returns.
#include <cstddef>

#include "dspark_common.cuh"
#include "host_util.cuh"
#include "sm100_ptx.cuh"
#include "tree_attention.cuh"

namespace dspark {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kTile = 128;             // keys of a tile
constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 bfloat16
constexpr int kNarrowRows = 32;        // rows that each warp of a stream has
constexpr uint32_t kSpin = 1u << 22;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.0f;         // log2 units that a weight may exceed 1

template <int D>
struct Shape {
  static constexpr int halves = D / 64;
  static constexpr int tile_bytes = halves * kHalfBytes;
  static constexpr int tiles = D == 128 ? 7 : 13;  // queries (1 or 2) and rings
  static constexpr uint32_t s_col(uint32_t i) { return 128 * i; }
  static constexpr uint32_t o_col(uint32_t i) { return 256 + D * i; }
  // Weights lie over the scores they come from, or, where tensor memory has
  // the room, apart: the next scores then need not wait for their product.
  static constexpr bool apart = D == 64;
  static constexpr uint32_t p_col(uint32_t i) { return apart ? 384 + 64 * i : s_col(i); }
};

// A unit as warp 2 describes it.
struct Unit {
  int n;            // its tiles here; 0: no more units
  int key;          // first key
  int s, len, cnt;  // sequence: its table row, committed and drafted tokens
  int b, h, t0;     // batch row, key head, first drafted token
  int both;         // more than 128 rows: half of them for each stream
  int whole;        // all of its tiles are here
};
constexpr int kUnits = 4, kUnitReaders = 11;  // warps 0, 1, 3 and the softmax

struct Control {  // shared memory behind the tiles
  // barriers: one arrival completes a phase of the first 31, four (a stream's
  // warps) one of those behind but v_all, which takes eight
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t q_full, q_empty, drain;
  uint64_t s_full[2], pv_done[2];  // of each stream
  uint64_t v_all, b_done;
  uint64_t p_ready[2], v_sync[2];  // of each stream
  // sums have been read: by the first stream at the end of every unit (both
  // streams' where it joins them), by the second where it has rows of its own.
  // Nobody arrives without work in the unit, so no phase is run ahead of.  The
  // products wait for them, and so does the second stream before it adds to its
  // sums by hand: a unit's first scores are there before the last unit's sums
  // have been read.
  uint64_t o_free[2];
  uint64_t u_full[kUnits], u_empty[kUnits];
  Unit units[kUnits];
  TreeShare share;
  uint32_t bad[2][4];     // rows of a value tile that hold NaN or infinities
  uint32_t add_first[2];  // the unit's first product adds to O
  float2 b_stats[128];    // the second stream's maximum and sum of each row
  uint32_t tmem;
  int failed;
};

template <int D>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)Shape<D>::tiles * Shape<D>::tile_bytes + sizeof(Control);
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory of a block");

// Narrow units: the weights of both streams, and what a stream's warps tell
// each other about each row.  Behind them there is always more shared memory
// that a product may read: it takes 128 rows of weights, of which 32 count.
struct Narrow {
  uint8_t weights[2][2][kNarrowRows * 128];  // [stream][64 keys]
  float top[2][4][kNarrowRows];              // of each warp: a maximum that raises m,
  float sum[2][4][kNarrowRows];              // and at the end its part of l
  uint32_t raise[2][4];                      // the warp has such maxima
  uint8_t rest[32768 - 16384 - 2048 - 32];
};
static_assert(sizeof(Narrow) == 32768, "a multiple of every tile");

// The polls of a wait that is not over at once: out of line, there are many.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity) {
  return mbar_wait(bar, parity, kSpin);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity);
}

// The same for a whole warp: either all its lanes go on or none does.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(bar, parity));
}

// Whether it is over, for a whole warp alike.
__device__ __forceinline__ bool over_warp(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done != 0);
}

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                       int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_5d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                       int x, int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v),
      "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#define R8(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), \
              "=r"(r[b + 5]), "=r"(r[b + 6]), "=r"(r[b + 7])
#define I8(b) "r"(r[b]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), \
              "r"(r[b + 5]), "r"(r[b + 6]), "r"(r[b + 7])

// 32 lanes x 32 columns, one lane of tensor memory a thread.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : R8(0), R8(8), R8(16), R8(24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::I8(0),
      I8(8), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : R8(0)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::I8(0),
               "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t at) {
  uint32_t x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void tmem_st1(uint32_t at, uint32_t x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(x), "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Which of the keys j .. j + 31 a row sees: committed ones lo .. len - 1, and
// drafted ones by their bits.
__device__ __forceinline__ uint32_t seen32(int j, int lo, int len, uint64_t bits) {
  const int a = lo - j, e = len - j;
  const uint32_t below = e <= 0 ? 0u : e >= 32 ? ~0u : (1u << e) - 1;
  const uint32_t under = a <= 0 ? 0u : a >= 32 ? ~0u : (1u << a) - 1;
  uint32_t m = below & ~under;
  if (e <= 0) {
    if (e > -64) m |= (uint32_t)(bits >> -e);
  } else if (e < 32) {
    m |= (uint32_t)(bits << e);
  }
  return m;
}

struct TcArgs {
  TreeArgs a;
  int page_rows;  // rows of a copy: of one page, at most a tile
  int pages;      // copies of half a tile
  int fit;        // drafted tokens of a stream's 128 rows
  int q_tokens;   // drafted tokens of a query copy
  int q_tiles;    // query tiles of a unit: 2 where units have more than 128 rows
  int k_slots, v_slots;  // tiles of the rings
  int page_shift;        // log2 of the page size
  int out32;             // out is aligned to 32 bytes
  int narrow;            // at most 32 rows a unit: the kernel's other form
  int stall;             // failure-path test: the product warp's wait runs out
};

// A role's place in a ring: the slot, and the parity of its phase.
struct Place {
  int slot;
  uint32_t parity;
  __device__ __forceinline__ void step(int slots) {
    if (++slot == slots) {
      slot = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A warp's view of the units.
struct UnitReader {
  Place at{0, 0};
  __device__ __forceinline__ bool next(Control& sh, Unit& u, bool& ok, int lane) {
    ok = wait_warp(&sh.u_full[at.slot], at.parity);
    if (!ok) return false;
    u = sh.units[at.slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.u_empty[at.slot]);
    at.step(kUnits);
    return u.n > 0;
  }
};

// 32 bytes in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// What hides keys from a row: see seen32.
struct Sight {
  int lo, len;
  uint64_t bits;
};

// The largest (c >= 0) or smallest (c < 0) score of the row that the thread
// holds, from tensor memory; hidden ones do not count.  Loops over parts of the
// row: code is slow the first time, when it comes from memory (20 cycles an
// instruction measured), and a block runs a few dozen tiles.
__device__ __forceinline__ float extreme_seen(uint32_t at, bool least, int j, const Sight& see) {
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    uint32_t x[32];
    tmem_ld32(at + 32 * h, x);
    const uint32_t w = seen32(j + 32 * h, see.lo, see.len, see.bits);
    tmem_ld_wait();
    if (least) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] ^= 0x80000000u;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float v = __uint_as_float(x[i]);
      if (!((w >> i) & 1)) v = -INFINITY;
      top[i & 1] = fmaxf(top[i & 1], v);
    }
  }
  const float best = fmaxf(top[0], top[1]);
  return least ? -best : best;
}

// Weights 2^(c s - base) of 32 scores, in bfloat16 to tensor memory; adds them
// to the sums in float32.  Hidden ones (0 in see) weigh nothing.
template <bool kMasked>
__device__ __forceinline__ void weigh32(uint32_t to, const uint32_t* x, uint32_t see, uint64_t cc,
                                        uint64_t bb, uint64_t (&sum)[2]) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 y = unpair(fma2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, bb));
    float p0 = ex2(y.x), p1 = ex2(y.y);
    if (kMasked) {
      p0 = (see >> (2 * i)) & 1 ? p0 : 0.0f;
      p1 = (see >> (2 * i)) & 2 ? p1 : 0.0f;
    }
    sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
    p[i] = pack_bf16(p0, p1);
  }
  tmem_st16(to, p);  // at most over scores that have been read
}

// The same over a whole row with hidden keys; returns the sum.
__device__ __forceinline__ float weigh_seen(uint32_t at, uint32_t to, float c, float base, int j,
                                            const Sight& see) {
  const uint64_t cc = pair(c, c), bb = pair(-base, -base);
  uint64_t sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    uint32_t x[32];
    tmem_ld32(at + 32 * h, x);
    const uint32_t w = seen32(j + 32 * h, see.lo, see.len, see.bits);
    tmem_ld_wait();
    weigh32<true>(to + 16 * h, x, w, cc, bb, sum);
  }
  const float2 t = unpair(add2(sum[0], sum[1]));
  return t.x + t.y;
}

// Narrow units: the two steps over the 32 scores that a warp has of its rows;
// the weights go to shared memory, half a row (64 keys) of 128 bytes whose
// 16-byte words are swizzled by the row.
__device__ __forceinline__ float extreme32(uint32_t (&x)[32], bool least, uint32_t see) {
  float top[2] = {-INFINITY, -INFINITY};
  const uint32_t flip = least ? 0x80000000u : 0u;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float v = __uint_as_float(x[i] ^ flip);
    top[i & 1] = fmaxf(top[i & 1], (see >> i) & 1 ? v : -INFINITY);
  }
  const float best = fmaxf(top[0], top[1]);
  return least ? -best : best;
}
__device__ __forceinline__ float weigh_narrow(uint8_t* to, int words, int swizzle,
                                              const uint32_t (&x)[32], uint32_t see, float c,
                                              float base) {
  const uint64_t cc = pair(c, c), bb = pair(-base, -base);
  uint64_t sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 8 * k + 2 * i;
      const float2 y = unpair(fma2(pair(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), cc, bb));
      float p0 = ex2(y.x), p1 = ex2(y.y);
      p0 = (see >> j) & 1 ? p0 : 0.0f;
      p1 = (see >> j) & 2 ? p1 : 0.0f;
      sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
      p[i] = pack_bf16(p0, p1);
    }
    *reinterpret_cast<uint4*>(to + (((4 * words + k) ^ swizzle) << 4)) =
        make_uint4(p[0], p[1], p[2], p[3]);
  }
  const float2 t = unpair(add2(sum[0], sum[1]));
  return t.x + t.y;
}

// Rows that see the whole tile: the same two steps, 64 scores at a time.
__device__ __forceinline__ float extreme_all(uint32_t at, bool least) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t x[64];
    tmem_ld32(at + 64 * h, x);
    tmem_ld32(at + 64 * h + 32, x + 32);
    tmem_ld_wait();
    if (least) {
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] ^= 0x80000000u;
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(x[i]));
  }
  const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  return least ? -best : best;
}

__device__ __forceinline__ float weigh_all(uint32_t at, uint32_t to, float c, float base) {
  const uint64_t cc = pair(c, c), bb = pair(-base, -base);
  uint64_t sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t x[64];
    tmem_ld32(at + 64 * h, x);
    tmem_ld32(at + 64 * h + 32, x + 32);
    tmem_ld_wait();
    weigh32<false>(to + 32 * h, x, 0, cc, bb, sum);
    weigh32<false>(to + 32 * h + 16, x + 32, 0, cc, bb, sum);
  }
  const float2 t = unpair(add2(sum[0], sum[1]));
  return t.x + t.y;
}

// The page numbers of a unit's tiles, 32 at a time: lane l has page first + l,
// or the place behind the pool, which reads as zeros.
struct Pages {
  const int32_t* row;  // of the block table
  int last;            // last page that holds a key of the sequence
  int first, ids;

  __device__ __forceinline__ int load(const TcArgs& P, int page) const {
    if (page > last) return P.a.c.num_pages;
    const int id = row[page];
    if (id >= 0 && id < P.a.c.num_pages) return id;
    cache_error(P.a.c, kCacheErrPage);
    return P.a.c.num_pages;
  }
  __device__ __forceinline__ void set(const TcArgs& P, const Unit& u, int lane) {
    row = P.a.c.block_table + (size_t)u.s * P.a.c.max_pages;
    last = (u.len + u.cnt - 1) >> P.page_shift;
    first = u.key >> P.page_shift;
    ids = load(P, first + lane);
  }
};

// The queries of a unit: one copy for each 128 rows and half of the head, or
// four of the same rows, one below the other, where units are narrow.
template <int D>
__device__ __forceinline__ void load_queries(const TcArgs& P, const Unit& u, const CUtensorMap* map,
                                             uint8_t* q_tile, uint64_t* full) {
  const int tiles = P.narrow ? 4 : 1 + u.both, copies = tiles * Shape<D>::halves;
  const int step = P.narrow ? kNarrowRows * 128 : Shape<D>::tile_bytes;
  mbar_arrive_expect_tx(full, copies * P.q_tokens * P.a.group * 128);
#pragma unroll 1
  for (int i = 0; i < copies; ++i) {
    const int tile = i / Shape<D>::halves, half = i - tile * Shape<D>::halves;
    tma_5d(q_tile + tile * step + half * kHalfBytes, map, full, half * 64, 0, u.h,
           P.narrow ? u.t0 : u.t0 + tile * P.fit, u.b);
  }
}

// Fills the ring of keys, or that of values and the queries before a unit's
// first values.
template <int D>
__device__ __noinline__ bool fill_ring(const TcArgs& P, Control& sh, bool values,
                                       const CUtensorMap* map, const CUtensorMap* map_q,
                                       uint8_t* q_tile, uint8_t* ring, int lane) {
  using S = Shape<D>;
  uint64_t* full = values ? sh.v_full : sh.k_full;
  uint64_t* empty = values ? sh.v_empty : sh.k_empty;
  const int slots = values ? P.v_slots : P.k_slots;
  Place at{0, 1};  // the phase that frees a slot: the first round passes
  int filled = 0, unit = 0;
  bool ok = true;
  // each lane copies one page's rows of one half of the head
  const int half = lane / P.pages, part = lane - half * P.pages;
  const bool mine = half < S::halves;
  uint8_t* const to = ring + half * kHalfBytes + part * P.page_rows * 128;
  UnitReader units;
  Unit next{}, cur{};
  Pages next_pages{}, pages{};
  bool some = units.next(sh, next, ok, lane);
  if (some && values && lane == 0)  // the first queries go before the pages are known
    load_queries<D>(P, next, map_q, q_tile, &sh.q_full);
  if (some) next_pages.set(P, next, lane);
#pragma unroll 1
  while (some && ok) {
    cur = next;
    pages = next_pages;
    if (values) {
      if (unit > 0) {
        ok = wait_warp(&sh.q_empty, (unit - 1) & 1);
        if (!ok) break;
        if (lane == 0) load_queries<D>(P, cur, map_q, q_tile, &sh.q_full);
        __syncwarp();
      }
      ++unit;
    }
    int ids2 = pages.load(P, pages.first + 32 + lane);
#pragma unroll 1
    for (int i = 0; i < cur.n; ++i) {
      const int j = cur.key + i * kTile, page = j >> P.page_shift;
      if (page >= pages.first + 32) {
        pages.first += 32;
        pages.ids = ids2;
        ids2 = pages.load(P, pages.first + 32 + lane);
      }
      ok = wait_warp(&empty[at.slot], at.parity);
      if (!ok) break;
      const int id = __shfl_sync(0xffffffffu, pages.ids, (page - pages.first + part) & 31);
      if (lane == 0) mbar_arrive_expect_tx(&full[at.slot], S::tile_bytes);
      __syncwarp();
      if (mine)
        tma_4d(to + at.slot * S::tile_bytes, map, &full[at.slot], half * 64,
               j & ((1 << P.page_shift) - 1), cur.h, id);
      at.step(slots);
      ++filled;
      if (i == 0) {  // the next unit, while this one's copies are under way
        some = units.next(sh, next, ok, lane);
        if (some) next_pages.set(P, next, lane);
        if (!ok) break;
      }
    }
  }
  if (!ok) {  // copies that nobody waited for land before the block ends
    for (int e = filled > slots ? filled - slots : 0; e < filled; ++e)
      wait_on(&full[e % slots], (e / slots) & 1);
    if (unit > 0) wait_on(&sh.q_full, (unit - 1) & 1);
  }
  return ok;
}

template <int D, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ TcArgs P, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v) {
  using S = Shape<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* q_tile = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Narrow& nar = *reinterpret_cast<Narrow*>(q_tile + P.q_tiles * S::tile_bytes);
  uint8_t* k_ring = q_tile + P.q_tiles * S::tile_bytes + (kNarrow ? sizeof(Narrow) : 0);
  uint8_t* v_ring = k_ring + P.k_slots * S::tile_bytes;
  Control& sh = *reinterpret_cast<Control*>(q_tile + S::tiles * S::tile_bytes);
  const TreeArgs& a = P.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // the next scores need not wait for the product of the weights
  constexpr bool apart = S::apart || kNarrow;
  static_assert(offsetof(Control, v_all) == 31 * 8 && offsetof(Control, o_free) == 37 * 8, "barriers");
  if (warp == 0) {
    uint64_t* bar = sh.k_full;
    mbar_init(bar + lane, lane < 31 ? 1 : 8);
    if (lane < 7) mbar_init(bar + 32 + lane, 4);
    if (lane < kUnits) {
      mbar_init(&sh.u_full[lane], 1);
      mbar_init(&sh.u_empty[lane], kUnitReaders);
    }
    if (lane < 2) sh.add_first[lane] = 0;
    if (lane == 0) sh.failed = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  follow();
  tc_fence_before();
  tree_start(a, sh.share);  // synchronises the block
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;

  if (warp == 0) {
    ok = fill_ring<D>(P, sh, false, &map_k, &map_q, q_tile, k_ring, lane);
  } else if (warp == 3) {
    ok = fill_ring<D>(P, sh, true, &map_v, &map_q, q_tile, v_ring, lane);
  } else if (warp == 1) {
    // -------------------------------------------------------- products
    // The whole warp runs this, so that descriptors stay in uniform
    // registers; one thread issues (issued from a single thread's code, each
    // product took 100 cycles to set up and bounded wide trees).
    const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
    const uint32_t idesc_o = idesc_bf16_f32(128, D, 0, 1);
    // keys and queries: rows of 128 bytes, 8-row groups 1024 bytes apart;
    // values: 64-wide halves kHalfBytes apart, 8-key groups 1024 bytes apart
    const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tile), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(k_ring), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(v_ring), kHalfBytes, 1024);
    const uint64_t p_desc = smem_desc_sw128(smem_u32(nar.weights), 16, 1024);
    uint32_t halved = 0, freed = 0;  // units that gave each stream half the rows
    uint32_t used[2] = {0, 0};       // tiles that a stream has weighed
    Place k{0, 0}, v{0, 0};
    // scores of the keys in k for a stream, from its query tile
    auto scores = [&](int st, int tile, bool free_keys, bool free_queries) {
      const uint64_t qd = q_desc + tile * (S::tile_bytes >> 4);
      const uint64_t kd = k_desc + k.slot * (S::tile_bytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i >> 2) * kHalfBytes + (i & 3) * 32) >> 4;
          mma_bf16(tmem + S::s_col(st), qd + off, kd + off, idesc_s, i != 0);
        }
        mma_commit(&sh.s_full[st]);
        if (free_keys) mma_commit(&sh.k_empty[k.slot]);
        if (free_queries) mma_commit(&sh.q_empty);
      }
      if (free_keys) k.step(P.k_slots);
    };
    auto keys = [&]() {
      ok = ok && wait_warp(&sh.k_full[k.slot], k.parity);
      tc_fence_after();
    };
    UnitReader units;
    Unit w;
#pragma unroll 1
    for (int unit = 0; ok && units.next(sh, w, ok, lane); ++unit) {
      ok = wait_warp(&sh.q_full, unit & 1);
      const bool both = !kNarrow && w.both;
      if (ok) keys();
      if (!ok) break;
      scores(0, 0, !both, w.n == 1 && !both);
      if (both) {
        scores(1, 1, true, w.n == 1);
      } else if (w.n > 1) {
        keys();
        if (!ok) break;
        scores(1, 0, true, w.n == 2);
      }
      if (unit > 0) ok = wait_warp(&sh.o_free[0], (unit - 1) & 1);
      if (freed < halved) ok = ok && wait_warp(&sh.o_free[1], freed++ & 1);
      halved += both;
      // failure-path test: scores are on their way, and nothing completes this
      // phase but the abort path itself
      if (P.stall) ok = __all_sync(0xffffffffu, ok && mbar_wait(&sh.drain, 0, kStallPolls));
      if (both && !apart) {  // bound by the products: as little as can be between them
#pragma unroll 1
        for (int i = 0; i < w.n && ok; ++i) {
          const bool more = i + 1 < w.n, last = i + 2 == w.n;
          ok = wait_warp(&sh.v_full[v.slot], v.parity);
          if (more) ok = ok && wait_warp(&sh.k_full[k.slot], k.parity);
          const uint64_t vd = v_desc + v.slot * (S::tile_bytes >> 4);
          const uint64_t kd = k_desc + k.slot * (S::tile_bytes >> 4);
          uint64_t* const v_empty = &sh.v_empty[v.slot];
          uint64_t* const k_empty = &sh.k_empty[k.slot];
          v.step(P.v_slots);
          if (more) k.step(P.k_slots);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait_warp(&sh.p_ready[h], used[h]++ & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t add = i > 0 || *(volatile uint32_t*)&sh.add_first[h];
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < kTile / 16; ++x)
                mma_bf16_ta(tmem + S::o_col(h), tmem + S::p_col(h) + 8 * x, vd + x * (2048 >> 4),
                            idesc_o, x != 0 ? 1u : add);
              mma_commit(&sh.pv_done[h]);
              if (more) {
                const uint64_t qd = q_desc + h * (S::tile_bytes >> 4);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                  const uint32_t off = ((x >> 2) * kHalfBytes + (x & 3) * 32) >> 4;
                  mma_bf16(tmem + S::s_col(h), qd + off, kd + off, idesc_s, x != 0);
                }
                mma_commit(&sh.s_full[h]);
                if (h == 1) mma_commit(k_empty);
                if (h == 1 && last) mma_commit(&sh.q_empty);
              }
              if (h == 1) mma_commit(v_empty);
            }
          }
        }
        continue;
      }
      if (kNarrow) {  // likewise
#pragma unroll 1
        for (int i = 0; i < w.n && ok; i += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (i + h >= w.n) break;
            const bool more = i + h + 2 < w.n;
            ok = ok && wait_warp(&sh.v_full[v.slot], v.parity);
            if (more) ok = ok && wait_warp(&sh.k_full[k.slot], k.parity);
            const uint64_t vd = v_desc + v.slot * (S::tile_bytes >> 4);
            const uint64_t kd = k_desc + k.slot * (S::tile_bytes >> 4);
            const uint64_t pd = p_desc + h * (sizeof(nar.weights[0]) >> 4);
            uint64_t* const v_empty = &sh.v_empty[v.slot];
            uint64_t* const k_empty = &sh.k_empty[k.slot];
            const bool last = i + h + 3 == w.n;
            v.step(P.v_slots);
            if (more) k.step(P.k_slots);
            ok = ok && wait_warp(&sh.p_ready[h], used[h]++ & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t add = i > 0 || *(volatile uint32_t*)&sh.add_first[h];
            if (elect_one()) {
              if (more) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                  const uint32_t off = ((x >> 2) * kHalfBytes + (x & 3) * 32) >> 4;
                  mma_bf16(tmem + S::s_col(h), q_desc + off, kd + off, idesc_s, x != 0);
                }
                mma_commit(&sh.s_full[h]);
                mma_commit(k_empty);
                if (last) mma_commit(&sh.q_empty);
              }
#pragma unroll
              for (int x = 0; x < kTile / 16; ++x)
                mma_bf16(tmem + S::o_col(h), pd + (((x >> 2) * kNarrowRows * 128 + (x & 3) * 32) >> 4),
                         vd + x * (2048 >> 4), idesc_o, x != 0 ? 1u : add);
              mma_commit(&sh.pv_done[h]);
              mma_commit(v_empty);
            }
          }
        }
      }
      if constexpr (!kNarrow) {
        auto weighed = [&](int st) {
          ok = ok && wait_warp(&sh.p_ready[st], used[st]++ & 1);
          tc_fence_after();
        };
        auto sums = [&](int st, bool first, bool free_values) {
          const uint32_t add = !first || *(volatile uint32_t*)&sh.add_first[st];
          const uint64_t vd = v_desc + v.slot * (S::tile_bytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i)
              mma_bf16_ta(tmem + S::o_col(st), tmem + S::p_col(st) + 8 * i, vd + i * (2048 >> 4),
                          idesc_o, i != 0 ? 1u : add);
            mma_commit(&sh.pv_done[st]);
            if (free_values) mma_commit(&sh.v_empty[v.slot]);
          }
        };
        for (int i = 0; i < w.n && ok; ++i) {
          // a stream's next scores go before its sums where the weights lie
          // apart, else behind them
          const bool more = i + (both ? 1 : 2) < w.n, last = i + (both ? 2 : 3) == w.n;
          bool there = false;  // the next keys
          for (int h = 0; h < (both ? 2 : 1) && ok; ++h) {
            const int st = both ? h : i & 1;
            auto next_scores = [&]() {
              if (h == 0 && !there) keys();  // both streams use the same ones
              if (ok) scores(st, both ? h : 0, !both || h == 1, last && (!both || h == 1));
            };
            if (h == 0) {  // behind the weights nothing should be waited for
              ok = wait_warp(&sh.v_full[v.slot], v.parity);
              there = more && over_warp(&sh.k_full[k.slot], k.parity);
            }
            weighed(st);
            if (apart && more && ok) next_scores();
            if (!ok) break;
            sums(st, i < (both ? 1 : 2), !both || h == 1);
            if (!apart && more) next_scores();
          }
          v.step(P.v_slots);
        }
      }
    }
    if (!ok) {
      if (elect_one()) mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, kSpin >> 4);
    }
  } else if (warp == 2) {
    // ----------------------------------------------------------- units
    if (lane == 0) {
      TreeWalk w = sh.share.walk;
      Place at{0, 1};
      bool some = w.n > 0, first = true;
#pragma unroll 1
      while (true) {
        ok = wait(&sh.u_empty[at.slot], at.parity);
        if (!ok) break;
        Unit u{};
        if (some) {
          u.n = w.n;
          u.key = (w.q.lo + w.first) * kTile;
          u.s = w.q.s;
          u.len = w.q.len;
          u.cnt = w.q.cnt;
          u.b = w.b;
          u.h = w.h;
          u.t0 = w.rt * a.row_tokens;
          u.both = w.q.cnt - u.t0 > P.fit;
          u.whole = w.whole;
        }
        sh.units[at.slot] = u;
        mbar_arrive(&sh.u_full[at.slot]);
        at.step(kUnits);
        if (first) tree_describe(a, w);
        first = false;
        if (!some) break;
        some = w.next(a);
      }
    }
  } else {
    // --------------------------------------------------------- softmax
    const int st = warp >= 8, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_at = lanes + S::o_col(st), p_real = lanes + S::p_col(st);
    const float c = a.scale * kLog2e;
    int g = 0, unit = 0;             // tiles of the units before, and those units
    uint32_t used = 0, syncs = 0, alls = 0, joins = 0;  // phases of the barriers
    bool is_first = true;            // the block's first unit
    // the row's token and head within a query tile
    const int row = kNarrow ? lane : r;
    const int r_token = (int)((uint32_t)row / (uint32_t)a.group), r_head = row - r_token * a.group;
    UnitReader units;
    // A unit, and what hides keys from this thread's row of it.  The next one's
    // is loaded before this one's results are written.
    struct View {
      Unit w;
      int t0, rows;
      Sight sight;
      int lo_most;  // committed keys below this are hidden from some row
    };
    auto look_at = [&](View& x) {
      const Unit& w = x.w;
      const int left = w.cnt - w.t0;
      x.t0 = w.t0 + (!kNarrow && w.both && st ? P.fit : 0);
      const int more = w.cnt - x.t0, tokens = more < P.fit ? more : P.fit;
      x.rows = tokens * a.group;
      const int t = x.t0 + r_token;
      const bool valid = row < x.rows;
      x.sight = Sight{valid ? tree_window_lo(a, w.b, t, w.len) : 0, w.len,
                      valid ? tree_mask(a, w.b, t, w.cnt) : 0};
      x.lo_most = 0;
      if (a.window > 0) {
        for (int i = lane; i < left && i < a.row_tokens; i += 32) {
          const int lo = tree_window_lo(a, w.b, w.t0 + i, w.len);
          x.lo_most = lo > x.lo_most ? lo : x.lo_most;
        }
      }
    };
    View cur, next;
    bool some = units.next(sh, cur.w, ok, lane);
    if (some) look_at(cur);
#pragma unroll 1
    for (; ok && some; g += cur.w.n, ++unit, cur = next) {
      const Unit& w = cur.w;
      const bool both = !kNarrow && w.both;       // half the rows each
      const int t0 = cur.t0, rows = cur.rows, t = t0 + r_token, len = w.len;
      // narrow: all warps weigh, the first one has the sums
      const bool valid = row < rows, any = kNarrow || quarter * 32 < rows;
      const bool sums = kNarrow ? quarter == 0 : any;
      const Sight sight = cur.sight;
      const int lo_most = a.window > 0 ? __reduce_max_sync(0xffffffffu, cur.lo_most) : 0;
      float m = -INFINITY, l = 0.0f;
      const int first = both ? 0 : st, step = both ? 1 : 2;
      // The block's first tile is rehearsed while its data are on their way:
      // the same code over whatever O holds, so that it is there when they
      // come.  O is this stream's own until its first weights are ready.
      bool real = is_first ? first >= w.n : true;
#pragma unroll 1
      for (int tile = first; tile < w.n && ok;) {
        const int j0 = w.key + tile * kTile;
        const bool masked = j0 + kTile > len || j0 < lo_most;
        const uint32_t s_at = lanes + (real ? S::s_col(st) : S::o_col(st));
        const uint32_t p_at = lanes + (real ? S::p_col(st) : S::o_col(st));
        if (real) {
          ok = wait_warp(&sh.s_full[st], used & 1);
          if (!ok) break;
        }
        tc_fence_after();
        if (any) {
          uint32_t x[32], see = ~0u;  // narrow: 32 scores of the row
          float best;
          if (kNarrow) {
            tmem_ld32(s_at + 32 * quarter, x);
            if (masked) see = seen32(j0 + 32 * quarter, sight.lo, sight.len, sight.bits);
            tmem_ld_wait();
            best = extreme32(x, c < 0.0f, see);
          } else {
            best = masked ? extreme_seen(s_at, c < 0.0f, j0, sight) : extreme_all(s_at, c < 0.0f);
          }
          best *= c;
          if (apart && used > 0 && real) {  // the last product has read its weights
            ok = wait_warp(&sh.pv_done[st], (used - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          const bool raise = valid && best > m + kRaise;  // m = -inf: any maximum
          uint32_t raised = __any_sync(0xffffffffu, raise);
          float now = raise ? best : m;
          if (kNarrow) {  // the warps agree
            if (raised) nar.top[st][quarter][lane] = now;
            if (lane == 0) nar.raise[st][quarter] = raised;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.v_sync[st]);
            ok = wait_warp(&sh.v_sync[st], syncs++ & 1);
            if (!ok) break;
            raised = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!*(volatile uint32_t*)&nar.raise[st][i]) continue;
              raised = 1;
              now = fmaxf(now, *(volatile float*)&nar.top[st][i][lane]);
            }
          }
          if (raised) {
            const float f = now != m ? ex2(m - now) : 1.0f;
            if (tile > first && sums) {  // the last product into O has ended
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) {
                uint32_t o[8];
                tmem_ld8(o_at + 8 * i, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st8(o_at + 8 * i, o);
              }
            }
            l *= f;
            m = now;
          }
          const float base = m == -INFINITY ? 0.0f : m;
          if (kNarrow) {
            l += weigh_narrow(nar.weights[st][quarter >> 1] + lane * 128, quarter & 1, lane & 7, x,
                              see, c, base);
            fence_proxy_async_smem();
          } else {
            l += masked ? weigh_seen(s_at, p_at, c, base, j0, sight) : weigh_all(s_at, p_at, c, base);
          }
          tmem_st_wait();
        }
        if (!real) {
          real = true;
          m = -INFINITY;
          l = 0.0f;
          continue;
        }
        uint32_t found = 0;
        if (masked) {
          // the tile's values: this thread looks through key j0 + r's
          const int round = (g + tile) / P.v_slots, slot = g + tile - round * P.v_slots;
          uint8_t* v = v_ring + slot * S::tile_bytes;
          ok = wait_warp(&sh.v_full[slot], round & 1);
          if (!ok) break;
          uint32_t worst = 0;
#pragma unroll
          for (int i = 0; i < S::halves * 8; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(
                v + (i >> 3) * kHalfBytes + r * 128 + (((i & 7) ^ (r & 7)) << 4));
            // an exponent of ones carries past it
            worst |= ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                     ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
          }
          const uint32_t b = __ballot_sync(0xffffffffu, (worst & 0x80008000u) != 0);
          if (lane == 0) {
            sh.bad[st][quarter] = b;
            mbar_arrive(&sh.v_sync[st]);
          }
          ok = wait_warp(&sh.v_sync[st], syncs++ & 1);
          if (!ok) break;
          uint32_t rows_bad[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            rows_bad[i] = *(volatile uint32_t*)&sh.bad[st][i];
            found |= rows_bad[i];
          }
          if (found) {
            if (st == 1 && tile == first && unit > 0) {
              // the first stream may still be reading the last unit's sums, its
              // join with these; it cannot end this unit before this stream has
              // gone on, so the phase is the last one or this one
              ok = wait_warp(&sh.o_free[0], (unit - 1) & 1);
              if (!ok) break;
              tc_fence_after();
            }
            if (sums) {
              if (tile == first) {  // O starts from what is added here
#pragma unroll 1
                for (int d = 0; d < D; ++d) tmem_st1(o_at + d, 0);
                tmem_st_wait();
              }
#pragma unroll 1
              for (int j = 0; j < kTile; ++j) {
                const uint32_t word = j < 64 ? (j < 32 ? rows_bad[0] : rows_bad[1])
                                             : (j < 96 ? rows_bad[2] : rows_bad[3]);
                if (!((word >> (j & 31)) & 1)) continue;
                uint32_t pp;
                if (kNarrow) {
                  pp = *reinterpret_cast<volatile uint32_t*>(
                      nar.weights[st][j >> 6] + lane * 128 + ((((j & 63) >> 3) ^ (lane & 7)) << 4) +
                      (j & 6) * 2);
                } else {
                  pp = tmem_ld1(p_real + (j >> 1));
                  tmem_ld_wait();
                }
                const float p = __uint_as_float(j & 1 ? pp & 0xffff0000u : pp << 16);
                const bool sees = seen32(j0 + j, sight.lo, sight.len, sight.bits) & 1;
#pragma unroll 1
                for (int d = 0; d < D; ++d) {
                  const uint16_t u = *reinterpret_cast<const uint16_t*>(
                      v + (d >> 6) * kHalfBytes + j * 128 + ((((d & 63) >> 3) ^ (j & 7)) << 4) + (d & 7) * 2);
                  if ((u & 0x7f80u) != 0x7f80u) continue;
                  const float o = __uint_as_float(tmem_ld1(o_at + d));
                  tmem_ld_wait();
                  tmem_st1(o_at + d, __float_as_uint(sees ? fmaf(p, bf16_bits_to_float(u), o) : o));
                  tmem_st_wait();
                }
              }
            }
            // cleared once every stream that uses the tile has read it, by one
            // of them, and used only then
            uint64_t* bar = both ? &sh.v_all : &sh.v_sync[st];
            uint32_t& phase = both ? alls : syncs;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            ok = wait_warp(bar, phase++ & 1);
            if (!ok) break;
            if ((!both || st == 0) && ((rows_bad[quarter] >> lane) & 1)) {
#pragma unroll 1
              for (int d = 0; d < D; ++d) {
                uint16_t* u = reinterpret_cast<uint16_t*>(
                    v + (d >> 6) * kHalfBytes + r * 128 + ((((d & 63) >> 3) ^ (r & 7)) << 4) + (d & 7) * 2);
                if ((*u & 0x7f80u) == 0x7f80u) *u = 0;
              }
            }
            fence_proxy_async_smem();
            if (both) {
              __syncwarp();
              if (lane == 0) mbar_arrive(bar);
              ok = wait_warp(bar, phase++ & 1);
              if (!ok) break;
            }
          }
        }
        if (quarter == 0 && lane == 0) *(volatile uint32_t*)&sh.add_first[st] = found != 0;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[st]);
        tile += step;
        ++used;
      }
      if (!ok) break;
      const bool worked = first < w.n;  // the stream had a tile of this unit
      some = units.next(sh, next.w, ok, lane);
      if (!ok) break;
      if (some) look_at(next);
      if (worked) {
        ok = wait_warp(&sh.pv_done[st], (used - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      if (kNarrow && worked) {
        nar.sum[st][quarter][lane] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_sync[st]);
        ok = wait_warp(&sh.v_sync[st], syncs++ & 1);
        if (!ok) break;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) l += *(volatile float*)&nar.sum[st][i][lane];
      }
      const int slot = 2 * blockIdx.x + (is_first ? 0 : 1);
      is_first = false;
      if (!both && st == 1) {
        // the first stream joins the two
        if (worked) {
          sh.b_stats[r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.b_done);
        }
      } else {
        const bool join = !both && w.n > 1;
        float fa = 1.0f, fb = 0.0f;
        if (join) {
          ok = wait_warp(&sh.b_done, joins++ & 1);
          if (!ok) break;
          tc_fence_after();
          const float2 o = sh.b_stats[r];
          const float now = fmaxf(m, o.x);
          fa = m == now ? 1.0f : ex2(m - now);
          fb = o.x == now ? 1.0f : ex2(o.x - now);
          l = l * fa + o.y * fb;
          m = now;
        }
        if (sums) {
          const size_t out_row = ((size_t)w.b * a.T + t) * a.heads + w.h * a.group + r_head;
          const int part_row = (t0 - w.t0) * a.group + row;
          const float inv = w.whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(o_at + 32 * i, o);
            if (join) {
              uint32_t o2[32];
              tmem_ld32(lanes + S::o_col(1) + 32 * i, o2);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * fa + __uint_as_float(o2[k]) * fb);
            } else {
              tmem_ld_wait();
            }
            if (valid && w.whole) {
              char* to = reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(a.out) + out_row * D + 32 * i);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t p[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                  p[d] = pack_bf16(__uint_as_float(o[16 * k + 2 * d]) * inv,
                                   __uint_as_float(o[16 * k + 2 * d + 1]) * inv);
                if (P.out32) {
                  store32(to + 32 * k, p);
                } else {
                  reinterpret_cast<uint4*>(to)[2 * k] = make_uint4(p[0], p[1], p[2], p[3]);
                  reinterpret_cast<uint4*>(to)[2 * k + 1] = make_uint4(p[4], p[5], p[6], p[7]);
                }
              }
            } else if (valid) {
              float* to = tree_part(a, slot) + (size_t)part_row * D + 32 * i;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t p[8];
#pragma unroll
                for (int d = 0; d < 8; ++d) p[d] = o[8 * k + d];
                store32(to + 8 * k, p);
              }
            }
          }
          if (valid) {
            if (!w.whole) {
              float* stats = tree_part_stats(a, slot) + 2 * part_row;
              stats[0] = m;
              stats[1] = l;
            } else if (a.lse) {
              a.lse[out_row] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && (both || st == 0)) mbar_arrive(&sh.o_free[st]);
    }
  }
  if (!ok) sh.failed = 1;
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sh.failed) cache_error(a.c, kDevErrTimeout);
}

bool is_power_of_two(int x) { return (x & (x - 1)) == 0; }

template <int D, bool kNarrow>
cudaError_t launch(const TreeArgs& a, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(tree_tc_kernel<D, kNarrow>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D>());
  if (e != cudaSuccess) return e;
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  TcArgs P{};
  P.a = a;
  P.page_rows = a.c.page_size < kTile ? a.c.page_size : kTile;
  P.pages = kTile / P.page_rows;
  P.fit = kTreeRows / a.group;
  P.q_tokens = a.T < P.fit ? a.T : P.fit;
  P.q_tiles = a.T > P.fit ? 2 : 1;
  P.narrow = kNarrow;
  P.stall = stall_first_wait_requested();
  const int slots = Shape<D>::tiles - P.q_tiles -
                    (kNarrow ? (int)sizeof(Narrow) / Shape<D>::tile_bytes : 0);
  P.v_slots = slots / 2;
  P.k_slots = slots - P.v_slots;
  while ((1 << P.page_shift) < a.c.page_size) ++P.page_shift;
  P.out32 = aligned_to(a.out, 32);
  CUtensorMap mq, mk, mv;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  {
    const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)a.group, (cuuint64_t)a.c.kv_heads,
                                (cuuint64_t)a.T, (cuuint64_t)a.B};
    const cuuint64_t row = (cuuint64_t)D * 2;
    const cuuint64_t strides[4] = {row, row * a.group, row * a.heads, row * a.heads * a.T};
    const cuuint32_t box[5] = {64, (cuuint32_t)a.group, 1, (cuuint32_t)P.q_tokens, 1};
    if (encode(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(a.q), dims, strides,
               box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    char* base = static_cast<char*>(a.c.pool) + cache_row(a.c, 2 * a.layer + i, 0, 0, 0);
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.c.page_size,
                                (cuuint64_t)a.c.kv_heads, (cuuint64_t)a.c.num_pages};
    const cuuint64_t row = (cuuint64_t)D * 2;
    const cuuint64_t strides[3] = {row, row * a.c.page_size, row * a.c.page_size * a.c.kv_heads};
    const cuuint32_t box[4] = {64, (cuuint32_t)P.page_rows, 1, 1};
    if (encode(i ? &mv : &mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return launch_behind(tree_tc_kernel<D, kNarrow>, a.blocks, kThreads, smem_bytes<D>(), stream, P, mq, mk, mv);
}

}  // namespace

bool tree_tc_supported(const TreeArgs& a) {
  return a.c.dtype == DSPARK_BF16 && (a.c.head_dim == 64 || a.c.head_dim == 128) &&
         a.c.page_size >= 8 && is_power_of_two(a.c.page_size);
}

cudaError_t launch_tree_tc(TreeArgs& a, int sms, cudaStream_t stream) {
  a.tile_shift = 7;
  static_assert(kTile == 1 << 7, "tile");
  const int fit = kTreeRows / a.group;  // tokens of a stream's rows
  a.row_tokens = a.T <= fit ? fit : 2 * fit;
  a.row_tiles = (a.T + a.row_tokens - 1) / a.row_tokens;
  a.slot_rows = (a.T < a.row_tokens ? a.T : a.row_tokens) * a.group;
  a.blocks = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
  const bool narrow = a.slot_rows <= kNarrowRows;
  if (a.c.head_dim == 64) return narrow ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  return narrow ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace dspark
