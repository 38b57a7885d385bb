// qt_mask_fp8.cu -- the query-tile kernel's masked fp8 instances (head_dim
// 128, 256), with a one-part or a two-part Q operand,
// with and without a softcap.
#include "decode_qt.cuh"

namespace kvq {

cudaError_t launch_qt_mask_fp8(int head_dim, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                                const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  return dispatch_qt_mask<KVQ_FP8_E4M3>(head_dim, split, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
