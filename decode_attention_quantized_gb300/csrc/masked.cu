// masked.cu -- the preparation of a masked call (kvq_attend_masked,
// kvq_key_mass): its virtual sequences and the key range that each of them
// needs, so that the split plan and the loads skip what no token sees.
#include "kvq_internal.h"
#include "ptx.cuh"
#include "score_rule.cuh"

namespace kvq {
namespace {

// One warp per group of T tokens: the union's bounds over its tokens.  Reads
// 8 bytes a token; a launch of its own because the groups' lengths are on the
// device and every CTA of the attention needs all of them for its plan.
__global__ void __launch_bounds__(256) vseq_kernel(const VSeqArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int v = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (v >= a.batch * a.n) return;
  const int b = v / a.n, j = v - b * a.n;
  const int lim = (a.max_seq_len > 0 && a.max_seq_len < a.cap) ? a.max_seq_len : a.cap;
  const int raw = a.seq_lens[b];
  if ((raw < 0 || raw > lim) && j == 0 && lane == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
  VSeq s;
  s.len = raw < 0 ? 0 : (raw > lim ? lim : raw);
  s.tok0 = b * a.C + j * a.T;
  s.ntok = min(a.T, a.C - j * a.T);
  s.pos0 = s.len - a.C + j * a.T;
  s.brow = b;
  // The union of the tokens' intervals: its hull [lo, hi), and whether every
  // interval touches the hull of those before it (then the hull has no gaps;
  // tokens of another order are taken to have some).
  int lo = 0x7FFFFFFF, hi = 0, gaps = 0;
  for (int i0 = 0; i0 < s.ntok; i0 += 32) {
    int begin = 0, end = 0;
    if (i0 + lane < s.ntok)
      dev::row_range(a.key_begin, a.key_end, a.window, (size_t)s.tok0 + i0 + lane, s.pos0 + i0 + lane, s.len, begin,
                     end);
    const bool some = begin < end;
    int pl = some ? begin : 0x7FFFFFFF, ph = some ? end : 0;  // inclusive scans over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int yl = __shfl_up_sync(0xffffffffu, pl, o), yh = __shfl_up_sync(0xffffffffu, ph, o);
      if (lane >= o) {
        pl = min(pl, yl);
        ph = max(ph, yh);
      }
    }
    int bl = __shfl_up_sync(0xffffffffu, pl, 1), bh = __shfl_up_sync(0xffffffffu, ph, 1);
    bl = lane == 0 ? lo : min(lo, bl);
    bh = lane == 0 ? hi : max(hi, bh);
    if (some && bh > 0 && (begin > bh || end < bl)) gaps = 1;
    lo = min(lo, __shfl_sync(0xffffffffu, pl, 31));
    hi = max(hi, __shfl_sync(0xffffffffu, ph, 31));
  }
  s.gaps = __any_sync(0xffffffffu, gaps);
  s.lo = hi > 0 ? lo : 0;
  s.hi = hi;
  if (lane == 0) a.out[a.by_group ? j * a.batch + b : v] = s;
}

// The keys of [0, len) that the key-mass kernel's pieces do not hold (below the
// first tile some token sees, or from `hi` on; every key when `all`): what
// they held before, decayed, 0 for the `fresh` last ones.
__global__ void __launch_bounds__(256) mass_rest_kernel(const DecodeArgs a, const MassArgs m, bool all) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int segs = a.batch * a.num_kv_heads;
  for (int seg = blockIdx.y; seg < segs; seg += gridDim.y) {
    const int b = seg / a.num_kv_heads, h = seg - b * a.num_kv_heads;
    const VSeq v = a.vseq[b];
    const int lo = v.lo & ~(m.tile - 1);
    const int32_t* bt = a.block_table + (size_t)v.brow * a.max_blocks_per_seq;
    for (int key = blockIdx.x * blockDim.x + threadIdx.x; key < v.len; key += gridDim.x * blockDim.x) {
      if (!all && key >= lo && key < v.hi) continue;
      const int id = bt[key >> a.log2_bs];
      if (id < 0 || id >= a.num_blocks) {
        atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
        continue;
      }
      float* p = m.mass + ((size_t)id * a.num_kv_heads + h) * a.block_size + (key & (a.block_size - 1));
      if (key >= v.len - m.fresh || m.decay == 0.0f) *p = 0.0f;
      else if (m.decay != 1.0f) *p = m.decay * *p;
    }
  }
}

}  // namespace

cudaError_t launch_mass_rest(const DecodeArgs& a, const MassArgs& m, bool all, int max_keys, cudaStream_t stream) {
  const int segs = a.batch * a.num_kv_heads;
  const unsigned y = (unsigned)(segs < 4096 ? segs : 4096);
  unsigned x = (unsigned)((max_keys + 1023) / 1024);
  if (x > 256) x = 256;
  return launch_pdl(mass_rest_kernel, dim3(x, y), 256, 0, stream, a, m, all);
}

cudaError_t launch_vseq(const VSeqArgs& a, cudaStream_t stream) {
  const long long warps = (long long)a.batch * a.n;
  return launch_pdl(vseq_kernel, (unsigned)((warps + 7) / 8), 256, 0, stream, a);
}

}  // namespace kvq
