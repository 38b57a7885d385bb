// key_mass_fp8.cu -- the key-mass kernel's fp8 instances.
#include "key_mass.cuh"

namespace kvq {

cudaError_t launch_key_mass_fp8(int head_dim, int nt, const CUtensorMap& tk, const DecodeArgs& a, const MassArgs& m,
                                 int grid, size_t smem, cudaStream_t stream) {
  return dispatch_key_mass<KVQ_FP8_E4M3>(head_dim, nt, a.k_mode, &tk, &a, &m, grid, smem, stream, nullptr);
}

cudaError_t occupancy_key_mass_fp8(int head_dim, int nt, int k_mode, size_t smem, int* blocks_per_sm) {
  return dispatch_key_mass<KVQ_FP8_E4M3>(head_dim, nt, k_mode, nullptr, nullptr, nullptr, 0, smem, nullptr,
                                     blocks_per_sm);
}

}  // namespace kvq
