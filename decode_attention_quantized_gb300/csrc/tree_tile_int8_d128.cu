// tree_tile_int8_d128.cu -- the tcgen05 draft-tree kernel's int8 instances for
// head_dim 128: a one-part or a two-part Q operand, rows once or folded, with
// and without a softcap.
#include "tree_tile.cuh"

namespace kvq {

cudaError_t launch_tree_tile_int8_d128(bool split, bool fold, const CUtensorMap& tk, const CUtensorMap& tv,
                                     const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  return dispatch_tree_tile<KVQ_INT8, 128>(split, fold, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
