// part_attention_tc.cu -- the attention of drafted tokens on the tensor cores
// over items (tree_attention_tc.cuh).
#include "tree_attention_tc.cuh"

namespace dspark {

cudaError_t launch_items_tc(const TreeArgs& a, cudaStream_t stream) {
  return launch_all<true>(a, stream);
}

cudaError_t launch_two_lines_tc(const TreeArgs& many, const TreeArgs& narrow, cudaStream_t stream) {
  return many.c.head_dim == 64 ? launch_two<64>(many, narrow, stream) : launch_two<128>(many, narrow, stream);
}

}  // namespace dspark
