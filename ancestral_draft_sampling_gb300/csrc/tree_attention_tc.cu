// tree_attention_tc.cu -- the attention of drafted tokens on the tensor cores
// over sequences (tree_attention_tc.cuh).
#include "tree_attention_tc.cuh"

namespace dspark {

bool tree_tc_supported(const TreeArgs& a) {
  const int page = a.c.page_size;
  return a.c.dtype == DSPARK_BF16 && (a.c.head_dim == 64 || a.c.head_dim == 128) && page >= 8 &&
         (page & (page - 1)) == 0;
}

bool tree_tc_narrow(const TreeArgs& a, int tokens) { return tokens * a.group <= kNarrowRows; }

void tree_tc_plan(TreeArgs& a, int tokens, int sms) {
  a.most = tokens;
  a.tile_shift = 7;
  static_assert(kTile == 1 << 7, "tile");
  const int fit = kTreeRows / a.group;  // tokens of a stream's rows
  a.row_tokens = tokens <= fit ? fit : 2 * fit;
  a.row_tiles = (tokens + a.row_tokens - 1) / a.row_tokens;
  a.slot_rows = (tokens < a.row_tokens ? tokens : a.row_tokens) * a.group;
  a.blocks = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
}

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
  return launch_all<false>(a, stream);
}

}  // namespace dspark
