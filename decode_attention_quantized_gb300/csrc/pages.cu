// pages.cu -- kvq_pages_step: block tables, the free list, slot map, positions
// and prefix sums of a step, from request lengths on the device.
//
// One thread plans up to kPerThread sequences: pages held and wanted, then two
// block-wide prefix sums (first over what is asked for, which settles the
// refusals, then over what is granted).  With them each page that changes hands
// and each new token is found on its own: the k-th page asked for is entry
// free_count + R - 1 - k of the stack on which the R given-back pages lie, and a
// token's sequence is found by bisection of the prefix sums.  Nothing depends
// on another CTA, so every CTA repeats the plan (B <= 1024: 12 KB of lengths
// from L2) and takes its share of tokens and pages.
//
// Bound: 16 bytes a token written, for prompts; for a decode step the latency
// of a dependent chain (lengths, two prefix sums, the page, the store).
#include "kvq_internal.h"
#include "ptx.cuh"

namespace kvq {
namespace {

constexpr int kPerThread = kMaxBatch / kPagesThreads;

struct PagesShared {
  int cu[kMaxBatch + 1];    // granted tokens before a sequence
  int pop[kMaxBatch + 1];   // granted pages before it
  int push[kMaxBatch + 1];  // given-back pages before it
  int start[kMaxBatch];
  int have[kMaxBatch];      // pages it holds
  int want[kMaxBatch];      // pages it has after the call
  long long warp_sum[kPagesThreads / 32][3];
};

// Exclusive prefix sums over the threads of N values each, and their totals.
template <int N, typename T>
__device__ __forceinline__ void block_scan(T (&v)[N], T (&total)[N], PagesShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T own[N];
#pragma unroll
  for (int i = 0; i < N; ++i) own[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T y = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += y;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) s.warp_sum[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w) {
      const T x = (T)s.warp_sum[w][i];
      if (w < warp) before += x;
      all += x;
    }
    v[i] = before + v[i] - own[i];
    total[i] = all;
  }
  __syncthreads();
}

// Last b with pre[b] <= x, for 0 <= x < pre[n] (sequences of nothing are skipped).
__device__ __forceinline__ int find(const int* pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// last: the launch that writes the lengths and the count.  Where these are
// written in place, every CTA has to have read them before, and more than one
// CTA takes a launch of its own for it; otherwise one launch does all.
__global__ void __launch_bounds__(kPagesThreads) pages_kernel(const PagesArgs a, bool rest, bool last) {
  __shared__ PagesShared s;
  // A launch that only commits reads its inputs at once: the one before it has
  // let it start after its own wait, so whatever wrote them has completed.
  if (rest) ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tid = threadIdx.x, B = a.batch, bs = a.block_size, cap = a.max_blocks_per_seq * bs;
  const bool first = blockIdx.x == 0 && rest;  // the CTA that flags
  unsigned int flags = 0;
  auto up = [&](int n) { return (n + bs - 1) >> a.log2_bs; };

  // ---- what each sequence asks for; a refusal for length or tokens
  int held[kPerThread], start[kPerThread], add[kPerThread];
  bool valid[kPerThread], ok[kPerThread];
  long long ask[2] = {0, 0}, sum[2];
  const int per = (B + kPagesThreads - 1) / kPagesThreads;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    valid[i] = false;
    held[i] = start[i] = add[i] = 0;
    if (i >= per || b >= B) continue;
    held[i] = a.held_lens[b];
    start[i] = a.start_lens ? a.start_lens[b] : held[i];
    add[i] = a.new_tokens[b];
    valid[i] = held[i] >= 0 && held[i] <= cap && start[i] >= 0 && start[i] <= held[i] && add[i] >= 0;
    if (!valid[i]) flags |= KVQ_DEVERR_SEQ_LEN;
  }
  int have[kPerThread], want[kPerThread];
  long long more[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    have[i] = valid[i] ? up(held[i]) : 0;
    // (start + add may pass 32 bits; such rows exceed the table row)
    ok[i] = valid[i] && (long long)start[i] + add[i] <= cap;
    if (valid[i] && !ok[i]) flags |= KVQ_DEVERR_SEQ_LEN;
    const long long w = ((long long)start[i] + add[i] + bs - 1) >> a.log2_bs;
    want[i] = ok[i] ? (int)w : have[i];
    more[i] = valid[i] && w > have[i] ? w - have[i] : 0;
    if (valid[i]) ask[0] += add[i];
    ask[1] += more[i];
  }
  block_scan(ask, sum, s);
  long long tokens = ask[0];
  long long back[1] = {0}, backs[1];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (!valid[i]) continue;
    tokens += add[i];
    if (add[i] > 0 && tokens > a.max_tokens) {
      flags |= KVQ_DEVERR_SEQ_LEN;
      ok[i] = false;
    }
    if (ok[i] && want[i] < have[i]) back[0] += have[i] - want[i];
  }
  block_scan(back, backs, s);
  int count = *a.free_count;
  if (count < 0 || count > a.num_blocks) {
    flags |= KVQ_DEVERR_BLOCK_ID;
    count = count < 0 ? 0 : a.num_blocks;
  }
  // (given-back pages past the pool's size are not taken)
  const int R = (int)(backs[0] > a.num_blocks - count ? a.num_blocks - count : backs[0]);
  if (backs[0] > R) flags |= KVQ_DEVERR_BLOCK_ID;
  const int supply = count + R;

  // ---- a refusal for pages; the prefix sums of what is granted
  long long asked = ask[1], got[3] = {0, 0, 0}, all[3];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    asked += more[i];
    if (ok[i] && more[i] > 0 && asked > supply) {
      flags |= KVQ_DEVERR_NO_BLOCKS;
      ok[i] = false;
    }
    if (!ok[i]) want[i] = have[i];
    if (ok[i]) {
      got[0] += add[i];
      if (want[i] > have[i]) got[1] += want[i] - have[i];
      if (want[i] < have[i]) got[2] += have[i] - want[i];
    }
  }
  block_scan(got, all, s);
  {
    long long t = got[0], p = got[1], q = got[2];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * per + i;
      if (i >= per || b >= B) continue;
      s.cu[b] = (int)t;
      s.pop[b] = (int)p;
      s.push[b] = (int)(q < R ? q : R);
      s.start[b] = start[i];
      s.have[b] = have[i];
      s.want[b] = want[i];
      if (ok[i]) {
        t += add[i];
        p += want[i] > have[i] ? want[i] - have[i] : 0;
        q += want[i] < have[i] ? have[i] - want[i] : 0;
      }
    }
  }
  const int n_tokens = (int)all[0], P = (int)all[1];
  if (tid == 0) {
    s.cu[B] = n_tokens;
    s.pop[B] = P;
    s.push[B] = R;
  }
  __syncthreads();

  // the k-th page that is asked for
  auto page = [&](int k) -> int {
    const int at = supply - 1 - k;
    if (at < count) return a.free_blocks[at];
    const int b = find(s.push, B, at - count);
    return a.block_table[(size_t)b * a.max_blocks_per_seq + s.want[b] + (at - count - s.push[b])];
  };
  const int top = B > 1 ? 1 << (31 - __clz(B - 1)) : 0;  // first step of a search over the sequences
  const int step = gridDim.x * kPagesThreads, id = blockIdx.x * kPagesThreads + tid;
  if (rest) {
    for (int k = id; k < P; k += step) {
      const int b = find(s.pop, B, k), pg = page(k);
      if (pg < 0 || pg >= a.num_blocks) flags |= KVQ_DEVERR_BLOCK_ID;
      a.block_table[(size_t)b * a.max_blocks_per_seq + s.have[b] + (k - s.pop[b])] = pg;
    }
    // what is left of the given-back pages (those below were popped again)
    for (int r = id; r < R - P; r += step) {
      const int pg = page(R - 1 - r);
      if (pg < 0 || pg >= a.num_blocks) flags |= KVQ_DEVERR_BLOCK_ID;
      a.free_blocks[count + r] = pg;
    }
    for (int i = id; i <= B; i += step) a.cu_seqlens[i] = s.cu[i];
    // four entries a thread at a time, side by side: an entry is a chain of two
    // searches and two reads
    for (int i0 = id; i0 < a.max_tokens; i0 += 4 * step) {
      int b[4], x[4], own[4], k[4], pg[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] = min(i0 + u * step, n_tokens - 1);  // (n_tokens - 1 may be -1: sequence 0, not used)
        b[u] = 0;
      }
      for (int w = top; w > 0; w >>= 1) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (b[u] + w < B && s.cu[b[u] + w] <= x[u]) b[u] += w;
      }
      // its page: one the sequence holds, or the k-th that is asked for
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] -= s.cu[b[u]];
        const int p = (s.start[b[u]] + x[u]) >> a.log2_bs;
        own[u] = p < s.have[b[u]] ? p : -1;
        k[u] = supply - 1 - (s.pop[b[u]] + p - s.have[b[u]]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        pg[u] = -1;
        if (i0 + u * step >= min(n_tokens, a.max_tokens)) continue;
        if (own[u] >= 0) pg[u] = a.block_table[(size_t)b[u] * a.max_blocks_per_seq + own[u]];
        else if (k[u] < count) pg[u] = a.free_blocks[k[u]];
        else pg[u] = page(supply - 1 - k[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * step;
        if (i >= a.max_tokens) continue;
        long long slot = -1, pos = 0;
        if (i < n_tokens) {
          const int row = s.start[b[u]] + x[u];
          if (pg[u] >= 0 && pg[u] < a.num_blocks) slot = ((long long)pg[u] << a.log2_bs) + (row & (bs - 1));
          else flags |= KVQ_DEVERR_BLOCK_ID;
          pos = row;
          if (a.parents && x[u] < a.tree_nodes) {
            const int32_t* up_of = a.parents + (size_t)b[u] * a.tree_nodes;
            int depth = 0;
            for (int n = x[u], m = up_of[n]; m >= 0 && m < n; n = m, m = up_of[n]) ++depth;
            pos = s.start[b[u]] + depth;
          }
        }
        a.slot_mapping[i] = slot;
        a.positions[i] = pos;
      }
    }
  }
  if (last) {
    if (!rest) ptx::griddep_wait();  // the launch before has read the lengths
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * per + i;
      if (blockIdx.x == 0 && i < per && b < B) a.seq_lens[b] = ok[i] ? start[i] + add[i] : held[i];
    }
    if (id == 0) *a.free_left = supply - P;
  }
  if (!first) flags &= KVQ_DEVERR_BLOCK_ID;  // the plan's flags are every CTA's
  if (rest && flags) atomicOr(a.err, flags);
}

}  // namespace

cudaError_t launch_pages_step(const PagesArgs& a, int sms, cudaStream_t stream) {
  // (1024 sequences taking in 212,000 tokens: 11.4 us in one launch, 13.1 with a
  // second one; 152 CTAs 13.3, 830 CTAs of one entry a thread 17.3: each repeats
  // the plan)
  const bool in_place = a.seq_lens == a.held_lens || a.seq_lens == a.start_lens || a.free_left == a.free_count;
  const int ctas = (a.max_tokens + 4 * kPagesThreads - 1) / (4 * kPagesThreads);
  const int grid = ctas <= 4 ? 1 : ctas < 4 * sms ? ctas : 4 * sms;
  if (grid == 1 || !in_place) return launch_pdl(pages_kernel, grid, kPagesThreads, 0, stream, a, true, true);
  if (cudaError_t e = launch_pdl(pages_kernel, grid, kPagesThreads, 0, stream, a, true, false)) return e;
  return launch_pdl(pages_kernel, 1, kPagesThreads, 0, stream, a, false, true);
}

}  // namespace kvq
