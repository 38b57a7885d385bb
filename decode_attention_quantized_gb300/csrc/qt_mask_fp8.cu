// qt_mask_fp8.cu -- the query-tile kernel's masked fp8 instances (head_dim
// 128, 256).
#include "decode_qt.cuh"

namespace kvq {

cudaError_t launch_qt_mask_fp8(int head_dim, const CUtensorMap& tk, const CUtensorMap& tv, const DecodeArgs& a,
                                int grid, size_t smem, cudaStream_t stream) {
  return dispatch_decode_qt<KVQ_FP8_E4M3, true>(head_dim, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
