// score_rule.cuh -- the score rule of the masked calls (kvq_score_mask): which
// keys a query row sees, and the distance bias its scores get.  Shared by the
// masked attention kernels, their combine and the key-mass kernel, so that all
// of them give a key of a row the same score.
#pragma once

#include "kvq_internal.h"

namespace kvq {
namespace dev {

// The score rule of one query row of a masked call (kvq_score_mask): the row
// sees keys of [begin, end), and a key at distance d = |pos - key| gets the
// bias ns * (d - d0) in log2 units, ns = -slope * log2 e.  d0 is the distance
// at which the row's largest bias over its keys falls (the nearest visible
// key's, the furthest one's when the slope is negative): taking it out leaves
// the softmax as it is and keeps the biases of the keys that matter near 0,
// where fp32 resolves them, however far from the query they lie; the combine
// puts ns * d0 back into the log-sum-exp.
struct __align__(16) RowRule {
  int begin, end, pos, d0;
  float ns;
  int bits;  // draft trees: where the row's bits begin in DecodeArgs::tree_bits (-1: none)
  int pad[2];
};

// The score x of `key` under a row's rule, key by key: the slow form, for
// tiles that some row does not see whole or that reach past a position.
__device__ __forceinline__ float rule_score(const RowRule& r, float x, int key, bool bias, bool& seen) {
  if (bias) x = fmaf(r.ns, (float)(abs(r.pos - key) - r.d0), x);
  seen = key >= r.begin && key < r.end;
  return seen ? x : -INFINITY;
}

// Draft trees: the row of a node sees the prefix keys [begin, end) and, of the
// nodes' keys from `end` on, those whose bit is set.
__device__ __forceinline__ bool tree_sees(const DecodeArgs& a, const RowRule& r, int key) {
  const int d = key - r.end;
  if (r.bits < 0 || (unsigned)d >= 32u * (unsigned)a.tree_words) return false;
  return (a.tree_bits[r.bits + (d >> 5)] >> (d & 31)) & 1u;
}

// The same for the 64 keys from key0 on, as bits.
__device__ __forceinline__ void tree_sees_64(const DecodeArgs& a, const RowRule& r, int key0, uint32_t (&m)[2]) {
  const int d = key0 - r.end, w0 = d >> 5;
  uint32_t w[3];
#pragma unroll
  for (int j = 0; j < 3; ++j)
    w[j] = r.bits >= 0 && (unsigned)(w0 + j) < (unsigned)a.tree_words ? a.tree_bits[r.bits + w0 + j] : 0u;
  m[0] = __funnelshift_r(w[0], w[1], (unsigned)d & 31u);
  m[1] = __funnelshift_r(w[1], w[2], (unsigned)d & 31u);
}

// rule_score for the instances of draft trees.
template <bool TREE>
__device__ __forceinline__ float row_score(const DecodeArgs& a, const RowRule& r, float x, int key, bool bias,
                                           bool& seen) {
  if constexpr (!TREE) return rule_score(r, x, key, bias, seen);
  seen = (key >= r.begin && key < r.end) || tree_sees(a, r, key);
  return seen ? x : -INFINITY;
}

// tok: index of the row's token in [B, C]; hi: one past the last key loaded.
// end is at most hi but may be any value below 0: compare it, subtract nothing
// from it (a RowRule's is cut).
__device__ __forceinline__ void row_range(const int32_t* key_begin, const int32_t* key_end, int window, size_t tok,
                                          int pos, int hi, int& begin, int& end) {
  begin = key_begin ? max(0, key_begin[tok]) : 0;
  if (window > 0 && pos >= window) begin = max(begin, pos - window + 1);
  end = min(key_end ? key_end[tok] : pos + 1, hi);
}

// The distance d0 of RowRule (0 for a row that sees nothing).
__device__ __forceinline__ int row_anchor(float slope, int pos, int begin, int end) {
  if (begin >= end) return 0;
  if (slope < 0.0f) return max(abs(pos - begin), abs(pos - (end - 1)));
  return pos < begin ? begin - pos : (pos >= end ? pos - (end - 1) : 0);
}

template <bool TREE = false>
__device__ __forceinline__ RowRule row_rule(const DecodeArgs& a, size_t tok, int pos, int hq, int hi) {
  RowRule r{};
  r.pos = pos;
  row_range(a.key_begin, a.key_end, a.window, tok, pos, hi, r.begin, r.end);
  // its distance to a tile stays inside int32 (cut here and not in row_range,
  // which costs the tile kernel 2% of a prompt of documents)
  r.end = max(0, r.end);
  r.ns = 0.0f;
  r.d0 = 0;
  if constexpr (TREE) {
    r.bits = (int)tok * a.tree_words;  // (at most 2^18 tokens of 8 words)
    return r;
  }
  if (a.slopes) {
    const float s = a.slopes[hq];
    r.ns = -s * 1.4426950408889634f;
    r.d0 = row_anchor(s, pos, r.begin, r.end);
  }
  return r;
}

}  // namespace dev
}  // namespace kvq
