// decode_tree_int4.cu -- the decode kernel's int4 instances for draft trees
// (an interval of the prefix and the bits of the nodes per row).
#include "decode.cuh"

namespace kvq {

// blocks_per_sm: the occupancy query instead of a launch.
cudaError_t dispatch_decode_tree_int4(int head_dim, int nt, const CUtensorMap* tk, const CUtensorMap* tv,
                                     const DecodeArgs* a, int grid, int threads, size_t smem, cudaStream_t stream,
                                     int* blocks_per_sm) {
  if (blocks_per_sm)
    return dispatch_decode<KVQ_INT4, true, 3>(head_dim, nt, nullptr, nullptr, nullptr, 0, threads, smem, nullptr,
                                             blocks_per_sm);
  return dispatch_decode<KVQ_INT4, false, 3>(head_dim, nt, tk, tv, a, grid, threads, smem, stream, nullptr);
}

}  // namespace kvq
