// key_mass_tc_int8.cu -- the tensor-memory key-mass kernel's int8 instances.
#include "key_mass_tc.cuh"

namespace kvq {

cudaError_t launch_key_mass_tc_int8(int head_dim, const CUtensorMap& tk, const DecodeArgs& a, const MassArgs& m,
                                    int nr, int grid, size_t smem, cudaStream_t stream) {
  return dispatch_key_mass_tc<KVQ_INT8>(head_dim, tk, a, m, nr, grid, smem, stream);
}

}  // namespace kvq
