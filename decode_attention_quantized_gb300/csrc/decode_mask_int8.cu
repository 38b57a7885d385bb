// decode_mask_int8.cu -- the decode kernel's masked instances for int8 cache
// codes (distance bias and an interval of keys per query token).
#include "decode.cuh"

namespace kvq {

// decode_split_int8.cu
cudaError_t dispatch_decode_split_int8(int head_dim, int nt, const CUtensorMap* tk, const CUtensorMap* tv,
                                       const DecodeArgs* a, int grid, int threads, size_t smem, cudaStream_t stream,
                                       int* blocks_per_sm);

cudaError_t launch_decode_mask_int8(int head_dim, int nt, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const DecodeArgs& a, int grid, int threads, size_t smem, cudaStream_t stream) {
  if (split) return dispatch_decode_split_int8(head_dim, nt, &tk, &tv, &a, grid, threads, smem, stream, nullptr);
  return dispatch_decode<KVQ_INT8, false, 1>(head_dim, nt, &tk, &tv, &a, grid, threads, smem, stream, nullptr);
}

cudaError_t occupancy_decode_mask_int8(int head_dim, int nt, bool split, int threads, size_t smem,
                                       int* blocks_per_sm) {
  if (split)
    return dispatch_decode_split_int8(head_dim, nt, nullptr, nullptr, nullptr, 0, threads, smem, nullptr,
                                      blocks_per_sm);
  return dispatch_decode<KVQ_INT8, true, 1>(head_dim, nt, nullptr, nullptr, nullptr, 0, threads, smem, nullptr,
                                            blocks_per_sm);
}

}  // namespace kvq
