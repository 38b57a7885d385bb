// qt_mask_int8.cu -- the query-tile kernel's masked int8 instances (head_dim
// 128, 256), with a one-part or a two-part Q operand.
#include "decode_qt.cuh"

namespace kvq {

cudaError_t launch_qt_mask_int8(int head_dim, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                                const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  if (split) return dispatch_decode_qt<KVQ_INT8, 2>(head_dim, tk, tv, a, grid, smem, stream);
  return dispatch_decode_qt<KVQ_INT8, 1>(head_dim, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
