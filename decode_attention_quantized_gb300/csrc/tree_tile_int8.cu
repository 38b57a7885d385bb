// tree_tile_int8.cu -- the tcgen05 draft-tree kernel's int8 instances (head_dim
// 128, 256), with a one-part or a two-part Q operand, with and without a
// softcap.
#include "tree_tile.cuh"

namespace kvq {

cudaError_t launch_tree_tile_int8(int head_dim, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                             const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  return dispatch_tree_tile<KVQ_INT8>(head_dim, split, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
