// prompt.cu -- kvq_attend_prompt: causal attention of packed prompts over
// their bf16 K and V.
#include <cuda_bf16.h>

#include "kvq_internal.h"
#include "ptx.cuh"

namespace kvq {
namespace {

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// One warp per (token, query head): each lane holds D / 32 channels, keys one
// after another.
template <int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const PromptArgs a) {
  constexpr int E = D / 32;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)a.total_tokens * a.num_q_heads;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
      const int s0 = a.cu_seqlens[b], s1 = a.cu_seqlens[b + 1];
      if (s0 < 0 || s1 < s0 || s1 > a.total_tokens || s1 - s0 > a.max_seq_len) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
    }
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
    const int t = (int)(r / a.num_q_heads), hq = (int)(r - (long long)t * a.num_q_heads), h = hq / a.group;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int s0 = a.cu_seqlens[lo], s1 = a.cu_seqlens[lo + 1];
    if (s0 < 0 || s1 < s0 || s1 > a.total_tokens || s1 - s0 > a.max_seq_len || t < s0 || t >= s1) continue;
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = bf16_at(a.q + t * a.q_stride + (long long)hq * D + lane + 32 * e);
      o[e] = 0.0f;
    }
    for (int j = a.window > 0 ? max(s0, t - a.window + 1) : s0; j <= t; ++j) {
      float x = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[e], bf16_at(a.k + j * a.k_stride + (long long)h * D + lane + 32 * e), x);
#pragma unroll
      for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
      x *= a.sm_scale;
      if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
      const float mn = fmaxf(m, x), c = expf(m - mn), p = expf(x - mn);
      m = mn;
      l = l * c + p;
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = fmaf(p, bf16_at(a.v + j * a.v_stride + (long long)h * D + lane + 32 * e), o[e] * c);
    }
    const float lse = m + logf(l);
    float f = 1.0f / l;
    if (a.head_sink) f /= 1.0f + expf(a.head_sink[hq] - lse);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const __nv_bfloat16 y = __float2bfloat16_rn(o[e] * f);
      a.out[r * D + lane + 32 * e] = *reinterpret_cast<const uint16_t*>(&y);
    }
    if (a.lse_out && lane == 0) a.lse_out[r] = lse;
  }
}

}  // namespace

cudaError_t launch_attend_prompt(const PromptArgs& a, int sms, cudaStream_t stream) {
  const long long blocks = ((long long)a.total_tokens * a.num_q_heads + 7) / 8;
  const int grid = (int)(blocks < 64LL * sms ? blocks : 64LL * sms);
  switch (a.head_dim) {
    case 64: return launch_pdl(prompt_rows_kernel<64>, grid, 256, 0, stream, a);
    case 128: return launch_pdl(prompt_rows_kernel<128>, grid, 256, 0, stream, a);
    default: return launch_pdl(prompt_rows_kernel<256>, grid, 256, 0, stream, a);
  }
}

}  // namespace kvq
