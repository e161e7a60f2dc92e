// part_attention.cuh -- the attention over part of the cache: the kernels that
// make the items (TreeItem) before it and join its results behind it.
#pragma once

#include "tree_attention.cuh"

namespace dspark {

// Lists of selected pages, made into one list of a sequence's key head: an item
// each.
struct SparseArgs {
  TreeArgs a;            // a.items, a.item_work, a.page_list, a.page_bits are made here
  const int32_t* pages;  // [B][lists][kv_heads][count]
  int count, lists;
  int room;              // places of an item's list
};
cudaError_t launch_sparse_items(const SparseArgs& a, cudaStream_t stream);

// Groups of sequences with a shared prefix: an item for each group's prefix, and
// one for what each sequence has behind it.  Both kinds are one line of tiles (two =
// 0), or two, in launches of their own, where one sequence's rows and a group's want
// different forms of the kernel.
struct PrefixArgs {
  TreeArgs shared, own;        // items, item_work and item_base are made here; own: if two
  const int32_t* group_start;  // [groups + 1]
  const int32_t* prefix;       // [groups]
  int groups, two;
  int32_t* group_of;           // [B] the item of a sequence's prefix, or -1
};
cudaError_t launch_prefix_items(const PrefixArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_join(const PrefixArgs& a, cudaStream_t stream);

}  // namespace dspark
