// decode_mask_fp8.cu -- the decode kernel's masked instances for fp8 cache
// codes (distance bias and an interval of keys per query token).
#include "decode.cuh"

namespace kvq {

cudaError_t launch_decode_mask_fp8(int head_dim, int nt, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const DecodeArgs& a, int grid, int threads, size_t smem, cudaStream_t stream) {
  return dispatch_decode<KVQ_FP8_E4M3, false, true>(head_dim, nt, &tk, &tv, &a, grid, threads, smem, stream, nullptr);
}

cudaError_t occupancy_decode_mask_fp8(int head_dim, int nt, int threads, size_t smem, int* blocks_per_sm) {
  return dispatch_decode<KVQ_FP8_E4M3, true, true>(head_dim, nt, nullptr, nullptr, nullptr, 0, threads, smem, nullptr,
                                               blocks_per_sm);
}

}  // namespace kvq
