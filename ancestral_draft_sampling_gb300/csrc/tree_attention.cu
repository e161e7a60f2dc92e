// tree_attention.cu -- the attention of drafted tokens on the FFMA units over
// sequences (tree_attention_ffma.cuh), and the merge of partial results.
#include "tree_attention_ffma.cuh"

namespace dspark {
namespace {

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

}  // namespace

void tree_ffma_plan(TreeArgs& a, int tokens, int sms) {
  a.most = tokens;
  a.tile_shift = a.c.head_dim > 128 ? 5 : 6;
  a.row_tokens = kRows / a.group;
  a.row_tiles = (tokens + a.row_tokens - 1) / a.row_tokens;
  a.slot_rows = (tokens < a.row_tokens ? tokens : a.row_tokens) * a.group;
  a.blocks = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
}

cudaError_t launch_tree_ffma(const TreeArgs& a, cudaStream_t stream) {
  return launch_ffma_all<false>(a, stream);
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
