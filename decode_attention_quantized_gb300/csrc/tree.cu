// tree.cu -- trees of drafted tokens: what each node sees of the cache
// (kvq_attend_tree's preparation), and the accepted path with the move of its
// rows (kvq_tree_accept).  Both read a few hundred integers a sequence and are
// bound by the latency of dependent reads, so a tree is read into shared memory
// once and walked there.
#include "kvq_internal.h"
#include "ptx.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 128;

// Rows of sequence b, and nodes among them; both cut to what they may be.
__device__ __forceinline__ void tree_size(const int32_t* seq_lens, const int32_t* num_nodes, int b, int lim, int T,
                                          int& len, int& n, bool& bad) {
  const int raw = seq_lens[b], nodes = num_nodes ? num_nodes[b] : T;
  len = min(max(raw, 0), lim);
  n = min(min(max(nodes, 0), T), len);
  bad = raw != len || nodes != n;
}

// One CTA per sequence.  A node's bits are those of the chain up from it; with
// a window W those of the W nearest of the chain, and of the prefix what the
// window leaves at the node's position.
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const TreeArgs a) {
  __shared__ int parent[KVQ_MAX_TREE_NODES];
  __shared__ int low[KVQ_MAX_TREE_NODES];  // first key a node needs
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, C = a.C;
  const int lim = (a.max_seq_len > 0 && a.max_seq_len < a.cap) ? a.max_seq_len : a.cap;
  int len, n;
  bool bad;
  tree_size(a.seq_lens, a.num_nodes, b, lim, C, len, n, bad);
  if (bad && tid == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
  for (int i = tid; i < n; i += kThreads) {
    const int p = a.parents[(size_t)b * C + i];
    parent[i] = p >= 0 && p < i ? p : -1;
  }
  __syncthreads();
  const int P = len - n;
  for (int i = tid; i < C; i += kThreads) {
    uint32_t w[KVQ_MAX_TREE_NODES / 32] = {};
    int depth = -1;
    if (i < n) {
      for (int m = i; m >= 0; m = parent[m]) {
        ++depth;
        if (a.window > 0 && depth >= a.window) continue;
#pragma unroll
        for (int j = 0; j < KVQ_MAX_TREE_NODES / 32; ++j)
          if (j == m >> 5) w[j] |= 1u << (m & 31);
      }
    }
    const size_t tok = (size_t)b * C + i;
#pragma unroll
    for (int j = 0; j < KVQ_MAX_TREE_NODES / 32; ++j)
      if (j < a.words) a.bits[tok * a.words + j] = w[j];
    const int begin = i < n && a.window > 0 ? max(0, P + depth - a.window + 1) : 0;
    a.begin[tok] = i < n ? begin : 0x7FFFFFFF;  // (no key; the attention kernel knows absent nodes by it)
    a.end[tok] = i < n ? P : 0;
    low[i] = min(begin, P);
  }
  __syncthreads();
  for (int j = tid; j < a.n; j += kThreads) {
    VSeq s;
    s.len = len;
    s.tok0 = b * C + j * a.T;
    s.ntok = min(a.T, C - j * a.T);
    s.pos0 = P + j * a.T;
    s.brow = b;
    const int real = min(s.ntok, n - j * a.T);
    int lo = P, all = 0;
    for (int i = 0; i < real; ++i) {
      lo = min(lo, low[j * a.T + i]);
      all = max(all, low[j * a.T + i]);
    }
    s.gaps = all;
    s.lo = real > 0 ? lo : 0;
    s.hi = real > 0 ? P + j * a.T + real : 0;
    a.out[b * a.n + j] = s;
  }
}

// One CTA per (sequence, kv head); each finds the path for itself (the walk
// takes the time of its length in shared-memory reads).
// The moves go downwards (path[i] >= i), so a chunk of the path whose rows are
// all read before any is written, chunk after chunk, never overwrites a row
// that a later one reads.
constexpr int kStage = 8192;                        // bytes of codes a chunk holds
constexpr int kStageRows = kStage / 32;             // rows it may have (a row of a side has 32 bytes or more)
constexpr int kMaxScales = 2 * (256 / 32) + 1;      // fp32 values beside a row

__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const AcceptArgs a) {
  __shared__ int child[KVQ_MAX_TREE_NODES];  // lowest child with the chosen token
  __shared__ int path[KVQ_MAX_TREE_NODES];
  __shared__ int count;
  __shared__ __align__(16) uint8_t stage[kStage];
  __shared__ float scales[kStageRows * kMaxScales / 4];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, T = a.T;
  int len, n;
  bool bad;
  tree_size(a.seq_lens, a.num_nodes, b, a.lim, T, len, n, bad);
  if (bad && h == 0 && tid == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
  const int P = len - n;
  const int64_t* drafts = a.drafts + (size_t)b * T;
  const int64_t* chosen = a.chosen + (size_t)b * T;
  for (int i = tid; i < n; i += kThreads) child[i] = T;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int p = a.parents[(size_t)b * T + i];
    // (atomics of a minimum: their order does not matter)
    if (p >= 0 && p < i && drafts[i] == chosen[p]) atomicMin(&child[p], i);
  }
  __syncthreads();
  if (tid == 0) {
    int m = 0;
    for (int i = n > 0 ? 0 : T; i < T; i = child[i]) path[m++] = i;
    count = m;
  }
  __syncthreads();
  const int m = count;
  if (h == 0) {
    for (int i = tid; i < T; i += kThreads) a.path[(size_t)b * T + i] = i < m ? path[i] : -1;
    if (tid == 0) {
      a.accepted[b] = m;
      a.new_lens[b] = P + m;
      a.next_tokens[b] = m > 0 ? chosen[path[m - 1]] : -1;
    }
  }

  // ---- the rows that move: from the first whose place changes on
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks_per_seq;
  const int pieces = a.row_bytes / 16;               // of one side of a row
  const int per_row = a.sides * pieces;
  const int nf = a.n_scale[0] + (a.sides == 2 ? a.n_scale[1] : 0) + (a.mass ? 1 : 0);
  const int most = min(kStage / 16 / per_row, nf > 0 ? (int)(sizeof(scales) / 4) / nf : KVQ_MAX_TREE_NODES);
  // index of (position, this head)'s row in the pool; -1: no such block
  auto row_at = [&](int pos) -> long long {
    const int id = bt[pos >> a.log2_bs];
    if (id < 0 || id >= a.num_blocks) return -1;
    return ((long long)id * a.num_kv_heads + h) * a.block_size + (pos & (a.block_size - 1));
  };
  // the f-th fp32 value beside a row
  auto scale_at = [&](long long row, int f) -> float* {
    if (f < a.n_scale[0]) return a.scale[0] + row * a.n_scale[0] + f;
    f -= a.n_scale[0];
    if (a.sides == 2 && f < a.n_scale[1]) return a.scale[1] + row * a.n_scale[1] + f;
    return a.mass + row;
  };
  int i0 = 0;
  while (i0 < m && path[i0] == i0) ++i0;
  for (; i0 < m; i0 += most) {
    const int rows = min(most, m - i0);
    for (int t = tid; t < rows * per_row; t += kThreads) {
      const int i = t / per_row, c = t - i * per_row, side = c >= pieces;
      const long long src = row_at(P + path[i0 + i]);
      if (src < 0) {
        atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
        continue;
      }
      *reinterpret_cast<uint4*>(stage + 16 * t) =
          *reinterpret_cast<const uint4*>(a.codes[side] + src * a.row_bytes + 16 * (c - side * pieces));
    }
    for (int t = tid; t < rows * nf; t += kThreads) {
      const int i = t / nf;
      const long long src = row_at(P + path[i0 + i]);
      if (src >= 0) scales[t] = *scale_at(src, t - i * nf);
    }
    __syncthreads();
    for (int t = tid; t < rows * per_row; t += kThreads) {
      const int i = t / per_row, c = t - i * per_row, side = c >= pieces;
      const long long src = row_at(P + path[i0 + i]), dst = row_at(P + i0 + i);
      if (dst < 0) atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
      if (src < 0 || dst < 0) continue;
      *reinterpret_cast<uint4*>(a.codes[side] + dst * a.row_bytes + 16 * (c - side * pieces)) =
          *reinterpret_cast<const uint4*>(stage + 16 * t);
    }
    for (int t = tid; t < rows * nf; t += kThreads) {
      const int i = t / nf;
      const long long src = row_at(P + path[i0 + i]), dst = row_at(P + i0 + i);
      if (src >= 0 && dst >= 0) *scale_at(dst, t - i * nf) = scales[t];
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_tree_rows(const TreeArgs& a, cudaStream_t stream) {
  return launch_pdl(tree_rows_kernel, a.batch, kThreads, 0, stream, a);
}

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  return launch_pdl(tree_accept_kernel, dim3((unsigned)a.batch, (unsigned)a.num_kv_heads), kThreads, 0, stream, a);
}

}  // namespace kvq
