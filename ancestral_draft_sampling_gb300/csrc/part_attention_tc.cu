// part_attention_tc.cu -- the attention of drafted tokens on the tensor cores
// over items (tree_attention_tc.cuh).
#include "tree_attention_tc.cuh"

namespace dspark {

cudaError_t launch_items_tc(const TreeArgs& a, cudaStream_t stream) {
  return launch_all<true>(a, stream);
}

}  // namespace dspark
