// part_attention_ffma.cu -- the attention of drafted tokens on the FFMA units
// over items (tree_attention_ffma.cuh).
#include "tree_attention_ffma.cuh"

namespace dspark {

cudaError_t launch_items_ffma(const TreeArgs& a, cudaStream_t stream) {
  return launch_ffma_all<true>(a, stream);
}

}  // namespace dspark
