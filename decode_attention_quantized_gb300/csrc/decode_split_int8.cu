// decode_split_int8.cu -- the masked int8 instances with a two-part Q operand (a
// per-channel K scale and an lse that is asked for).
#include "decode.cuh"

namespace kvq {

// blocks_per_sm: the occupancy query instead of a launch.
cudaError_t dispatch_decode_split_int8(int head_dim, int nt, const CUtensorMap* tk, const CUtensorMap* tv,
                                       const DecodeArgs* a, int grid, int threads, size_t smem, cudaStream_t stream,
                                       int* blocks_per_sm) {
  if (blocks_per_sm)
    return dispatch_decode<KVQ_INT8, true, 2>(head_dim, nt, nullptr, nullptr, nullptr, 0, threads, smem, nullptr,
                                              blocks_per_sm);
  return dispatch_decode<KVQ_INT8, false, 2>(head_dim, nt, tk, tv, a, grid, threads, smem, stream, nullptr);
}

}  // namespace kvq
