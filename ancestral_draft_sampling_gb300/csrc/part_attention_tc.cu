// part_attention_tc.cu -- the attention of drafted tokens on the tensor cores
// over items (tree_attention_tc.cuh).
#include "tree_attention_tc.cuh"

namespace dspark {

// Heads of fewer dims than the kernel's are filled up with zeros by the copies, which
// costs products and no bytes (96 dims against the FFMA kernel: 22 x 8 tokens with lists
// of 32 pages 51 and 400 us, 44 single tokens behind a prefix 79 and 589, 16 x 8 tokens
// behind one of 16000 keys 62 and 1613; 16 dims, the first of these: 41 and 229).  The
// weights are rounded to bfloat16 with it, which the FFMA kernel does not do.
bool items_tc_supported(const TreeArgs& a) {
  const int page = a.c.page_size;
  return a.c.dtype == DSPARK_BF16 && a.c.head_dim <= 128 && a.c.head_dim % 16 == 0 && page >= 8 &&
         (page & (page - 1)) == 0;
}

cudaError_t launch_items_tc(const TreeArgs& a, cudaStream_t stream) {
  return launch_all<true>(a, stream);
}

}  // namespace dspark
