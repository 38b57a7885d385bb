// prompt.cu -- kvq_attend_prompt: causal attention of packed prompts over
// their bf16 K and V, on the tcgen05 tensor cores.
//
// Mathematics: for a row (token i, query head) S_j = sm_scale <q, k_j> (capped)
// over the keys j <= i (and j > i - window) of its sequence; with a running
// reference mu and P_j = 2^(S_j log2 e - mu): o = sum P_j v_j / sum P_j, lse =
// ln 2 (mu + log2 sum P_j).
//
// A tile is 128 rows: the G query heads of a kv head times tpt = 128 / G tokens
// (row = token x G + head), so that the heads of a group share their K and V.
// A work unit is one or two (head_dim 64, 128) tiles of one kv head that follow
// one another, run against the sequence's key tiles of 128 keys:
//
//   S [128 rows x 128 keys] = Q [128 x D] . K [128 x D]^T   A = Q, B = K (shared, K-major)
//   O [128 rows x D]     (+)= P [128 x 128] . V [128 x D]    A = P (TMEM), B = V (shared, MN-major)
//
// P overwrites its own S in tensor memory.  With two tiles the MMAs of one run
// while the softmax of the other works; head_dim 256 has one tile and two S
// buffers, for the same reason.  K and V tiles come through a ring of TMA
// stages of 128 keys x (up to) 128 channels; Q by one TMA box of G heads x tpt
// tokens per 64 channels.
//
// Warps: softmax, one thread a row, four warps per tile (S out of tensor
// memory, mask, lazy reference maxima -- O is rescaled only when a row's
// maximum grows by more than 2^8 --, P back; at the end O, normalised, to
// memory); then one producer (work units, TMA) and one MMA warp.
//
// A weight of 0 times infinity or NaN is NaN, so a V row may spoil the rows of a
// tile that do not see it.  A unit whose results hold NaN therefore runs again
// with care: in key tiles that some row does not see whole, elements of V that
// are not finite are set to 0 before the product, and rows that see them get
// them added at the end.  It costs a barrier, a look at the results and longer
// code: one prompt of 77 tokens 5.4 -> 5.8 us, 64 of 200 tokens 77 -> 83, 16,384
// tokens 1%.  (Two warps that look through those tiles every time: 5.7, 85 and the
// same, but 185 -> 200 us with a window of 1024 at head_dim 256.)
#include <cuda_bf16.h>

#include "decode_tc.cuh"

namespace kvq {
namespace {

constexpr int kKeys = 128;           // keys per tile
constexpr int kSlab = kKeys * 128;   // bytes of 64 channels of a tile
constexpr int kSmallBatch = 64;      // sequences whose units a warp finds without a plan

template <int D_>
struct PromptCfg {
  static constexpr int D = D_;
  static constexpr int NQ = D == 256 ? 1 : 2;      // row tiles of a unit
  static constexpr int SB = D == 256 ? 2 : 1;      // S buffers of a tile
  static constexpr int NH = D == 256 ? 2 : 1;      // stages of a K or V tile
  static constexpr int SD = D < 128 ? D : 128;     // channels of a stage
  static constexpr int STAGE = SD / 64 * kSlab;
  static constexpr int QTILE = D / 64 * kSlab;
  static constexpr int STAGES = D == 64 ? 8 : 5;
  static constexpr int SOFTMAX = 4 * NQ;           // warps
  static constexpr int THREADS = 32 * (SOFTMAX + 4);  // (a whole warpgroup beside the softmax: register shares)
  static constexpr int O_COL = 256;
  // shared memory behind the 1 KB alignment: Q, ring, barriers, units
  static constexpr int RING = NQ * QTILE;
  static constexpr int BARS = RING + STAGES * STAGE;
  static constexpr int N_BARS = 2 * STAGES + 2 * NQ + 3 * NQ * SB + NQ + 4;
  static constexpr int UNITS = BARS + (N_BARS * 8 + 15) / 16 * 16;
  static constexpr int TOTAL = UNITS + 2 * 16 + 16 + 8 * 4;
  static constexpr int SMEM = TOTAL + 1024;
};

// One unit's rows and keys.  Token 0 of the unit is token q0 of the sequence,
// whose rows begin at row0.
struct __align__(16) Unit {
  int row0, len, q0, head;  // len 0: the last units are done; -1: nothing to do
};
constexpr int kCare = 1 << 30;  // in head: the unit runs again, with care for V

// The key tiles [a, b) that tile w of a unit needs.
struct Range {
  int a, b;
};
__device__ __forceinline__ Range tile_range(const Unit& u, int w, int tpt, int window) {
  const int t0 = u.q0 + w * tpt, t1 = min(t0 + tpt, u.len);
  if (t0 >= t1) return {0, 0};
  return {window > 0 ? max(0, t0 - window + 1) / kKeys : 0, (t1 - 1) / kKeys + 1};
}

// Every row of a unit of `tokens` tokens sees all of the key tiles [a, b) that it
// multiplies; of the others some row may not see some key.
__device__ __forceinline__ Range whole_range(const Unit& u, int tokens, int window) {
  const int last = min(u.q0 + tokens, u.len) - 1;
  return {window > 0 ? (max(0, last - window + 1) + kKeys - 1) / kKeys : 0, (u.q0 + 1) / kKeys};
}

__device__ __forceinline__ bool bad_bounds(const PromptArgs& a, int s0, int s1) {
  return s0 < 0 || s1 < s0 || s1 > a.total_tokens || s1 - s0 > a.max_seq_len;
}
// Where bounds descend, a sequence may also begin before the end of an earlier
// one; it is skipped, so that no row is written for two sequences and the work is
// that of at most total_tokens.  (One that descends is among the flagged.)

// The plan of many units: [0] the next unit, [1] blocks of tokens in all, then
// for the sequences in order of length, longest first, the prefix sums of
// their blocks [B + 1], their first rows [B] and lengths [B].
__global__ void __launch_bounds__(1024) prompt_plan_kernel(const PromptArgs a, int unit_tokens, int grid) {
  __shared__ int len[kMaxBatch], sorted[kMaxBatch], sums[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5, B = a.batch;
  int s0 = 0, n = 0;
  bool descends = false;
  if (b < B) {
    s0 = a.cu_seqlens[b];
    const int s1 = a.cu_seqlens[b + 1];
    descends = s1 < s0;
    const bool bad = bad_bounds(a, s0, s1);
    if (bad) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
    else n = s1 - s0;
    len[b] = n;
    sorted[b] = bad ? 0 : s1;
  }
  if (__syncthreads_or(descends)) {
    for (int i = 0; i < b && b < B; ++i)
      if (s0 < sorted[i]) n = 0;
    __syncthreads();
    if (b < B) len[b] = n;
    __syncthreads();
  }
  if (b < B) {
    int rank = 0;
    for (int i = 0; i < B; ++i) rank += len[i] > n || (len[i] == n && i < b);
    sorted[rank] = n;
    a.plan[2 + B + 1 + rank] = s0;
    a.plan[2 + 2 * B + 1 + rank] = n;
  }
  __syncthreads();
  int x = b < B ? (sorted[b] + unit_tokens - 1) / unit_tokens : 0;
  const int own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += sums[w];
  if (b < B) a.plan[2 + b] = x - own;
  if (b == B - 1) {
    a.plan[0] = grid;  // (each CTA has its first unit by its index)
    a.plan[1] = x;
    a.plan[2 + B] = x;
  }
}

// Unit u of the plan; a whole warp.
__device__ __forceinline__ Unit planned_unit(const PromptArgs& a, int u, int unit_tokens) {
  const int B = a.batch, lane = threadIdx.x & 31;
  const int* pre = a.plan + 2;
  const int blk = u / a.num_kv_heads;
  if (blk >= a.plan[1]) return {0, 0, 0, 0};
  // the last s with pre[s] <= blk, 32 at a time (pre[B] > blk)
  int i = lane * 32;
  const int hi = __popc(__ballot_sync(0xffffffffu, i < B && pre[i] <= blk)) - 1;
  i = hi * 32 + lane;
  const int s = hi * 32 + __popc(__ballot_sync(0xffffffffu, i < B && pre[i] <= blk)) - 1;
  Unit r;
  r.row0 = a.plan[2 + B + 1 + s];
  r.len = a.plan[2 + 2 * B + 1 + s];
  // the last tokens first: their rows see the most keys
  r.q0 = (pre[s + 1] - 1 - blk) * unit_tokens;
  r.head = u - blk * a.num_kv_heads;
  return r;
}

// Unit u of few sequences, straight from their bounds; a whole warp.
__device__ __forceinline__ Unit small_unit(const PromptArgs& a, int u, int unit_tokens) {
  const int lane = threadIdx.x & 31;
  int blk = u / a.num_kv_heads;
  const int head = u - blk * a.num_kv_heads;
  int ends = 0;  // the furthest end so far
  bool descends = false;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int s0 = 0, s1 = 0, n = 0;
    if (b0 + lane < a.batch) {
      s0 = a.cu_seqlens[b0 + lane];
      s1 = a.cu_seqlens[b0 + lane + 1];
      if (!bad_bounds(a, s0, s1)) n = s1 - s0;
      else if (u == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
    }
    int end = bad_bounds(a, s0, s1) ? 0 : s1;
    descends = __any_sync(0xffffffffu, descends || s1 < s0);
    if (descends || b0 > 0) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(0xffffffffu, end, o));
      const int up = __shfl_up_sync(0xffffffffu, end, 1);
      if (s0 < max(ends, lane > 0 ? up : 0)) n = 0;
      ends = max(ends, __shfl_sync(0xffffffffu, end, 31));
    } else if (b0 + 32 < a.batch) {
      ends = __reduce_max_sync(0xffffffffu, end);
    }
    const int own = (n + unit_tokens - 1) / unit_tokens;
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x > blk);
    if (hit) {
      const int s = __ffs(hit) - 1;
      Unit r;
      r.row0 = __shfl_sync(0xffffffffu, s0, s);
      r.len = __shfl_sync(0xffffffffu, n, s);
      r.q0 = (__shfl_sync(0xffffffffu, x, s) - 1 - blk) * unit_tokens;
      r.head = head;
      if (u != 0) return r;
      // (the flags of the sequences behind)
      for (int b = b0 + 32 + lane; b < a.batch; b += 32)
        if (bad_bounds(a, a.cu_seqlens[b], a.cu_seqlens[b + 1])) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
      return r;
    }
    blk -= __shfl_sync(0xffffffffu, x, 31);
  }
  return {0, 0, 0, 0};
}

// unit_tiles: row tiles of a unit (at most NQ; 1 when that fills the GPU
// better); planned: units by plan and counter, else one unit per CTA.
template <int D, bool CAP>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptArgs a, int unit_tiles, bool planned) {
  using C = PromptCfg<D>;
  constexpr int kProducer = C::SOFTMAX, kMma = C::SOFTMAX + 1;
  constexpr int NQ = C::NQ, SB = C::SB, NH = C::NH;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_base = ptx::smem_u32(base), ring = q_base + C::RING;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(base + C::BARS);  // [STAGES] stage landed
  uint64_t* bar_empty = bar_full + C::STAGES;                        // [STAGES] its MMAs complete
  uint64_t* b_qfull = bar_empty + C::STAGES;                         // [NQ] the unit's Q landed
  uint64_t* b_qfree = b_qfull + NQ;                                  // [NQ] its last QK^T complete
  uint64_t* b_s = b_qfree + NQ;                                      // [NQ][SB] S written
  uint64_t* b_p = b_s + NQ * SB;                                     // [NQ][SB][2] a half of P written, O rescaled
  uint64_t* b_o = b_p + 2 * NQ * SB;                                    // [NQ] a PV complete
  uint64_t* b_unit = b_o + NQ;                                       // [2] unit written
  uint64_t* b_ufree = b_unit + 2;                                    // [2] unit read
  Unit* units = reinterpret_cast<Unit*>(base + C::UNITS);            // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(units + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* total = abort_flag + 1;  // number of the unit behind the last one
  volatile int* spoilt = reinterpret_cast<volatile int*>(tmem_slot + 4);  // [8] at unit n & 7: n + 1, if it is to run again

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      ptx::mbar_init(&bar_full[i], 1);
      ptx::mbar_init(&bar_empty[i], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      ptx::mbar_init(&b_qfull[i], 1);
      ptx::mbar_init(&b_qfree[i], 1);
      ptx::mbar_init(&b_o[i], 1);
    }
    for (int i = 0; i < NQ * SB; ++i) {
      ptx::mbar_init(&b_s[i], 1);
      ptx::mbar_init(&b_p[2 * i], 4);
      ptx::mbar_init(&b_p[2 * i + 1], 4);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&b_unit[i], 1);
      ptx::mbar_init(&b_ufree[i], C::SOFTMAX + 1);
    }
    for (int i = 0; i < 8; ++i) spoilt[i] = 0;
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMma) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ptx::mbar_try_wait(bar, parity) || *abort_flag) return;
    if (!ptx::mbar_wait_bounded_inl(bar, parity)) {
      *abort_flag = 1;
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    }
  };
  const int G = a.group, tpt = 128 / G, W = a.window;
  // The units of this CTA, one after another, as the producer writes them.
  int un = 0;
  auto next_unit = [&]() -> Unit {
    wait(&b_unit[un & 1], (un >> 1) & 1);
    Unit u = units[un & 1];
    if (*abort_flag) u.len = 0;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&b_ufree[un & 1]);
    ++un;
    return u;
  };
  // Whether units follow behind one of len 0: the last two may have to run again.
  // (The same for every warp, whatever else has happened: nothing of it is written
  // again before all have read it.)
  auto go_on = [&]() -> bool {
    constexpr uint32_t kThreads = (C::SOFTMAX + 2) * 32;
    __syncwarp();
    ptx::named_bar_sync(1, kThreads);
    const int n = *total;
    const bool more = (n > 0 && spoilt[(n - 1) & 7] == n) || (n > 1 && spoilt[(n - 2) & 7] == n - 1);
    if (more) {
      __syncwarp();
      ptx::named_bar_sync(1, kThreads);
    }
    return more;
  };
  auto range = [&](const Unit& u, int w) -> Range {
    return w < unit_tiles ? tile_range(u, w, tpt, W) : Range{0, 0};
  };

  // 384 threads x 168 registers: the softmax holds a row of 128 scores
  constexpr bool kShares = NQ > 1;
  if (warp == kProducer) {
    // ============================================================ producer
    if constexpr (kShares) ptx::regs_down<88>();
    const int unit_tokens = unit_tiles * tpt;
    uint32_t slot = 0, phase = 0, issued = 0;
    int qn[NQ] = {};
    // one stage: `keys` rows of 128 keys from row z on, channels from x on
    auto load = [&](const CUtensorMap* tm, int x, int head, int z) {
      if (issued >= (uint32_t)C::STAGES) wait(&bar_empty[slot], phase ^ 1u);
      if (*abort_flag) return;
      ptx::mbar_arrive_expect_tx(&bar_full[slot], C::STAGE);
#pragma unroll
      for (int c = 0; c < C::SD / 64; ++c)
        ptx::tma_load_3d(ring + slot * C::STAGE + c * kSlab, tm, x + 64 * c, head, z, &bar_full[slot]);
      ++issued;
      if (++slot == C::STAGES) {
        slot = 0;
        phase ^= 1u;
      }
    };
    int u = blockIdx.x;
    Unit ahead{}, before[3] = {};  // the next unit; the last three written
    bool have = false;
    int late = 0;  // units that are looked after behind the list's end
    for (int n = 0;; ++n) {
      if (!have) {
        ahead = planned ? planned_unit(a, u, unit_tokens) : (u >= 0 ? small_unit(a, u, unit_tokens) : Unit{});
        have = true;
      }
      // Once unit n - 2 has been taken, unit n - 3 is finished: it may have to run
      // again.  The last two are looked after behind the end of the list.
      int again = 0;
      if (lane == 0 && n >= 2) {
        wait(&b_ufree[n & 1], ((n - 2) >> 1) & 1);
        again = n >= 3 && spoilt[(n - 3) & 7] == n - 2;
      }
      again = __shfl_sync(0xffffffffu, again, 0);
      Unit x = ahead;
      if (again) {
        x = before[2];
        x.head |= kCare;
      } else if (late > 0) {
        x.len = -1;
      } else {
        have = x.len == 0;
      }
      late = max(0, late - 1);
      before[2] = before[1];
      before[1] = before[0];
      before[0] = x;
      if (lane == 0) {
        units[n & 1] = x;
        x.head &= ~kCare;
        ptx::mbar_arrive(&b_unit[n & 1]);
        if (x.len > 0) {
          const Range r0 = range(x, 0), r1 = NQ > 1 ? range(x, NQ - 1) : Range{0, 0};
          const int end = max(r0.b, r1.b);
          auto load_q = [&](int w) {
            if (qn[w] > 0) wait(&b_qfree[w], (qn[w] - 1) & 1);
            if (*abort_flag) return;
            ptx::mbar_arrive_expect_tx(&b_qfull[w], (uint32_t)(D / 64) * 128u * (uint32_t)(G * tpt));
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              ptx::tma_load_3d(q_base + w * C::QTILE + c * kSlab, &tmq, 64 * c, x.head * G, x.row0 + x.q0 + w * tpt,
                               &b_qfull[w]);
            ++qn[w];
          };
          auto load_kv = [&](const CUtensorMap* tm, int j) {
#pragma unroll
            for (int h = 0; h < NH; ++h) load(tm, h * C::SD, x.head, x.row0 + j * kKeys);
          };
          load_q(0);
          load_kv(&tmk, r0.a);
          if (NQ > 1 && r1.b > 0) load_q(NQ - 1);
          // in the order of the MMAs below
          for (int j = r0.a; j < end; ++j) {
            if (NQ > 1) {
              load_kv(&tmv, j);
              if (j + 1 < end) load_kv(&tmk, j + 1);
            } else {
              if (j + 1 < end) load_kv(&tmk, j + 1);
              load_kv(&tmv, j);
            }
          }
        }
      }
      __syncwarp();
      if (x.len == 0 || *abort_flag) {
        if (x.len != 0 && lane == 0) {
          // a wait gave up: the others leave at the next unit, which is none
          units[(n + 1) & 1] = Unit{};
          ptx::mbar_arrive(&b_unit[(n + 1) & 1]);
        }
        // every copy has landed before the CTA may end
        if (lane == 0) {
          *total = n;
          const uint32_t last = issued < (uint32_t)C::STAGES ? issued : (uint32_t)C::STAGES;
          for (uint32_t i = issued - last; i < issued; ++i)
            ptx::mbar_wait_bounded_inl(&bar_full[i % C::STAGES], (i / C::STAGES) & 1);
          for (int w = 0; w < NQ; ++w)
            if (qn[w] > 0) ptx::mbar_wait_bounded_inl(&b_qfull[w], (qn[w] - 1) & 1);
        }
        if (!go_on()) break;
        late = 2;
      }
      if (!have) {
        if (lane == 0) u = planned ? atomicAdd(&a.plan[0], 1) : -1;
        u = __shfl_sync(0xffffffffu, u, 0);
      }
    }
  } else if (warp == kMma) {
    // ================================================================ MMA
    if constexpr (kShares) ptx::regs_down<88>();
    constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(128, kKeys);
    constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, C::SD) | (1u << 16);  // B MN-major
    const uint64_t kd = ptx::smem_desc_sw128(ring);
    const uint32_t k_lo = (uint32_t)kd, hi = (uint32_t)(kd >> 32);
    const uint32_t q_lo = (uint32_t)ptx::smem_desc_sw128(q_base);
    const uint32_t v_lo = (uint32_t)ptx::smem_desc_sw128_mn(ring, kSlab);
    uint32_t it = 0;               // stages taken from the ring
    uint32_t ns[NQ] = {};          // QK^Ts of a tile
    uint32_t np[NQ] = {};          // its PVs
    int qn[NQ] = {};
    auto stage_of = [&](uint32_t i) { return i % (uint32_t)C::STAGES; };
    auto landed = [&](uint32_t i) { wait(&bar_full[stage_of(i)], (i / (uint32_t)C::STAGES) & 1); };
    // QK^T of tile w with the K tile in stages i ..
    auto qk = [&](int w, uint32_t i) {
      const uint32_t buf = ns[w] % SB;
      __syncwarp();
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint32_t st = stage_of(i + c / (C::SD / 64)) * C::STAGE + (c % (C::SD / 64)) * kSlab;
        ptx::mma_f16_ss_x4(tmem + 128 * (w * SB + buf), q_lo + ((w * C::QTILE + c * kSlab) >> 4), k_lo + (st >> 4), hi,
                           idesc_qk, c > 0 ? 1u : 0u);
      }
      ptx::mma_commit(&b_s[w * SB + buf]);
      ++ns[w];
    };
    // PV of tile w with the V tile in stages i ..; the unit's first overwrites O
    auto pv = [&](int w, uint32_t i, bool first) {
      const uint32_t buf = np[w] % SB;
      const uint32_t p = tmem + 128 * (w * SB + buf);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        wait(&b_p[2 * (w * SB + buf) + half], (np[w] / SB) & 1);
        __syncwarp();
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < NH; ++h)
          ptx::mma_f16_ts_x4_step(tmem + C::O_COL + w * D + h * C::SD, p + 32 * half, 8,
                                  v_lo + ((stage_of(i + h) * C::STAGE + half * 64 * 128) >> 4), (16 * 128) >> 4, hi, idesc_pv,
                                  first && half == 0 ? 0u : 1u);
      }
      ptx::mma_commit(&b_o[w]);
      ++np[w];
    };
    auto release = [&](uint32_t i) {
#pragma unroll
      for (int h = 0; h < NH; ++h) ptx::mma_commit(&bar_empty[stage_of(i + h)]);
    };
    auto land = [&](uint32_t i) {
#pragma unroll
      for (int h = 0; h < NH; ++h) landed(i + h);
    };
    // Rows of V behind the sequence hold anything (NaN times a weight of 0 is
    // NaN): they are set to 0.  With care, elements before them that are not
    // finite are, too.
    auto clear = [&](uint32_t i, int rows, bool care) {
      for (int h = 0; h < NH; ++h) {
        const uint32_t st = ring + stage_of(i + h) * C::STAGE;
        for (int c = 0; c < C::SD / 64; ++c)
          for (int k = lane + (care ? 0 : 8 * rows); k < 8 * kKeys; k += 32) {
            const uint32_t at = st + c * kSlab + 16 * k;
            uint32_t x[4] = {0u, 0u, 0u, 0u};
            if (k < 8 * rows) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((x[e] & 0x7F80u) == 0x7F80u) x[e] &= 0xFFFF0000u;
                if ((x[e] & 0x7F800000u) == 0x7F800000u) x[e] &= 0xFFFFu;
              }
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
    };
    for (;;) {
      const Unit u = next_unit();
      if (u.len == 0) {
        // every MMA has completed before tensor memory can be released
        for (int w = 0; w < NQ; ++w)
          if (np[w] > 0 && !ptx::mbar_wait_bounded_inl(&b_o[w], (np[w] - 1) & 1) && lane == 0) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
        if (!go_on()) break;
      }
      if (u.len <= 0) continue;
      const Range whole = whole_range(u, unit_tiles * tpt, W);
      auto prepare = [&](uint32_t i, int j) {
        const bool care = (u.head & kCare) && (j < whole.a || j >= whole.b);
        if (care || (j + 1) * kKeys > u.len) clear(i, min(kKeys, u.len - j * kKeys), care);
      };
      const Range r0 = range(u, 0), r1 = NQ > 1 ? range(u, NQ - 1) : Range{0, 0};
      const int end = max(r0.b, r1.b);
      auto q_ready = [&](int w) {
        wait(&b_qfull[w], qn[w] & 1);
        ++qn[w];
      };
      uint32_t k_at = it, v_at;
      land(k_at);
      q_ready(0);
      qk(0, k_at);
      if (r0.a + 1 == r0.b) ptx::mma_commit(&b_qfree[0]);
      if (NQ > 1 && r1.b > 0) {
        q_ready(NQ - 1);
        if (r1.a <= r0.a) {
          qk(NQ - 1, k_at);
          if (r0.a + 1 == r1.b) ptx::mma_commit(&b_qfree[NQ - 1]);
        }
      }
      release(k_at);
      for (int j = r0.a; j < end; ++j) {
        const bool more = j + 1 < end;
        if (NQ > 1) {
          v_at = k_at + NH;
          k_at = v_at + NH;
          land(v_at);
          prepare(v_at, j);
          if (j < r0.b) pv(0, v_at, j == r0.a);
          if (more) {
            land(k_at);
            if (j + 1 < r0.b) {
              qk(0, k_at);
              if (j + 2 == r0.b) ptx::mma_commit(&b_qfree[0]);
            }
          }
          if (j >= r1.a && j < r1.b) pv(NQ - 1, v_at, j == r1.a);
          release(v_at);
          if (more) {
            if (j + 1 >= r1.a && j + 1 < r1.b) {
              qk(NQ - 1, k_at);
              if (j + 2 == r1.b) ptx::mma_commit(&b_qfree[NQ - 1]);
            }
            release(k_at);
          }
          it = v_at + NH;
        } else {
          if (more) {
            k_at += NH + (j > r0.a ? NH : 0);  // (the V tile of j - 1 lies between)
            land(k_at);
            qk(0, k_at);
            if (j + 2 == end) ptx::mma_commit(&b_qfree[0]);
            release(k_at);
            v_at = k_at + NH;
          } else {
            v_at = k_at + (j > r0.a ? 2 * NH : NH);
          }
          land(v_at);
          prepare(v_at, j);
          pv(0, v_at, j == r0.a);
          release(v_at);
          it = v_at + NH;
        }
      }
    }
  } else if (warp < C::SOFTMAX) {
    // ============================================================ softmax
    if constexpr (kShares) ptx::regs_up<208>();
    const int w = warp >> 2, q = warp & 3, r = 32 * q + lane;  // tile, row
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t o_col = t_lane + C::O_COL + w * D;
    const int t_row = dev::div_small(r, __frcp_rn((float)G)), g = r - t_row * G;
    // (finite and above 0, so that alpha times -inf is -inf)
    const float alpha = fminf(fmaxf(CAP ? a.sm_scale / a.softcap : a.sm_scale * kLog2e, 1.17549435e-38f), 3.4028234e38f);
    const float cap2 = CAP ? a.softcap * kLog2e : 0.0f;
    const dev::CapNear cap_near(cap2, alpha);
    const ptx::f32x2 aa = ptx::pack_x2(alpha, alpha);
    // (coefficients far from fp32's ends, or not at all)
    const float reach =
        CAP && alpha > 6e-5f && alpha < 1.6e4f && cap2 > 1e-6f && cap2 < 1e6f ? dev::CapNear::kReach / alpha : -1.0f;
    uint32_t ns = 0;  // S tiles taken
    for (;;) {
      Unit u = next_unit();
      if (u.len == 0 && !go_on()) break;
      const bool care = u.head & kCare;
      u.head &= ~kCare;
      const Range kr = u.len > 0 ? range(u, w) : Range{0, 0};
      if (kr.a >= kr.b) continue;
      const int tok = u.q0 + w * tpt + t_row;
      const bool valid = t_row < tpt && tok < u.len;
      const int pos = min(tok, u.len - 1), begin = W > 0 ? pos - W + 1 : 0;
      const bool idle = !__any_sync(0xffffffffu, valid);
      float mu = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      for (int j = kr.a; j < kr.b; ++j, ++ns) {
        const uint32_t buf = ns % SB;
        const uint32_t s_col = t_lane + 128 * (w * SB + buf);
        wait(&b_s[w * SB + buf], (ns / SB) & 1);
        if (idle) {  // rows of no token: what they hold is read by nobody
          if (lane == 0) {
            ptx::mbar_arrive(&b_p[2 * (w * SB + buf)]);
            ptx::mbar_arrive(&b_p[2 * (w * SB + buf) + 1]);
          }
          continue;
        }
        ptx::tc_fence_after();
        const int key0 = j * kKeys;
        const bool full = key0 + kKeys - 1 <= pos && key0 >= begin;
        const int lo = begin - key0, hi = pos - key0;  // the tile's visible keys
        // Scores of 128 keys in registers; under a cap, whose unrolled code would
        // not stay in the instruction cache, 32 at a time, twice.
        constexpr int CH = CAP ? 32 : kKeys;
        float y[CH];
        auto load_s = [&](int c0) {
          uint32_t v[CH];
#pragma unroll
          for (int c = 0; c < CH; c += 32) ptx::tmem_ld32(s_col + c0 + c, v + c);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            asm volatile("" : "+r"(v[i]));
            y[i] = __uint_as_float(v[i]);
          }
        };
        auto hide = [&](int c0) {
#pragma unroll
          for (int k = 0; k < CH; ++k)
            if (c0 + k < lo || c0 + k > hi) y[k] = -INFINITY;
        };
        float m = -INFINITY, least = INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < kKeys; c0 += CH) {
          load_s(c0);
          if (!full) hide(c0);
          float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY}, mn[4] = {least, INFINITY, INFINITY, INFINITY};
#pragma unroll
          for (int k = 0; k < CH; k += 2) {
            mx[k / 2 % 4] = ptx::max3(mx[k / 2 % 4], y[k], y[k + 1]);
            if constexpr (CAP) mn[k / 2 % 4] = ptx::min3(mn[k / 2 % 4], y[k], y[k + 1]);
          }
          m = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
          if constexpr (CAP) least = fminf(ptx::min3(mn[0], mn[1], mn[2]), mn[3]);
        }
        // Under a cap, tanh by the polynomial below where no score of the row
        // passes its reach (the usual scores), else by the quotient.
        const bool near = CAP && fmaxf(fabsf(m), fabsf(least)) <= reach;
        if constexpr (CAP) {
          if (near) {
            m = cap_near.score(m);
          } else if (m != -INFINITY) {
            float x[2] = {m * alpha, 0.0f};
            dev::cap_scores<2>(x, cap2);
            m = x[0];
          }
        } else {
          m *= alpha;
        }
        // move the reference only when the tile's maximum exceeds it by more
        // than 8; a row with no key yet holds zeros in O
        float corr = 1.0f;
        bool resc = false;
        if (m > mu + 8.0f) {
          if (mu != -INFINITY) {
            corr = ptx::fast_exp2(mu - m);
            resc = true;
          }
          mu = m;
        }
        l0 *= corr;
        l1 *= corr;
        const float nmu = mu == -INFINITY ? 0.0f : -mu;
        if (__any_sync(0xffffffffu, resc)) {
          wait(&b_o[w], (ns - 1) & 1);  // the PV before (a rescale is never a unit's first tile)
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            dev::tmem_ld_cols<16>(o_col + c0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= corr;
            dev::tmem_st_cols<16>(o_col + c0, o);
          }
        }
        // P = 2^(y - mu), bf16 pairs; the sums take the fp32 weights.  P goes out
        // in two halves: PV over the first runs while the second is computed.
        const ptx::f32x2 nm = ptx::pack_x2(nmu, nmu);
        ptx::f32x2 l = ptx::pack_x2(l0, l1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[kKeys / 4];
          // the weights of y[at ..] into p[to ..]
          auto weigh = [&](int at, int to, int n, auto&& score) {
#pragma unroll
            for (int i = 0; i < n; i += 2) {
              float z0, z1;
              ptx::unpack_x2(score(ptx::pack_x2(y[at + i], y[at + i + 1])), z0, z1);
              const float e0 = ptx::fast_exp2(z0), e1 = ptx::fast_exp2(z1);
              l = ptx::add_x2(l, ptx::pack_x2(e0, e1));
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
              p[to + i / 2] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          };
          if constexpr (!CAP) {
            weigh(half * (kKeys / 2), 0, kKeys / 2, [&](ptx::f32x2 x) { return ptx::fma_x2(x, aa, nm); });
            ptx::tmem_st32(s_col + 32 * half, p);
          } else {
#pragma unroll 1
            for (int c0 = half * (kKeys / 2); c0 < (half + 1) * (kKeys / 2); c0 += CH) {
              load_s(c0);
              if (near) {
                // (a row with hidden keys, of score -inf, is not near)
                weigh(0, 0, CH, [&](ptx::f32x2 x) { return cap_near.scores(x, nm); });
              } else {
#pragma unroll
                for (int k = 0; k < CH; k += 2) ptx::mul_x2(y[k], y[k + 1], y[k], y[k + 1], alpha, alpha);
                dev::cap_scores<CH>(y, cap2);
                if (!full) hide(c0);
                weigh(0, 0, CH, [&](ptx::f32x2 x) { return ptx::add_x2(x, nm); });
              }
              // (the columns of S that P takes have been read: P is half as wide)
              __syncwarp();
              ptx::tmem_st16(s_col + c0 / 2, *reinterpret_cast<uint32_t(*)[16]>(p));
            }
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&b_p[2 * (w * SB + buf) + half]);
        }
        ptx::unpack_x2(l, l0, l1);
      }
      // ---- O of the unit, normalised, to memory
      if (SB > 1 && kr.b - kr.a > 1) wait(&b_o[w], (ns - 2) & 1);  // (phases one at a time)
      wait(&b_o[w], (ns - 1) & 1);
      if (idle) continue;
      ptx::tc_fence_after();
      const float l = l0 + l1;
      const int hq = u.head * G + g;
      const size_t row = (size_t)(u.row0 + (valid ? tok : 0)) * a.num_q_heads + (valid ? hq : 0);
      const float lse = (mu + ptx::fast_log2(l)) * 0.69314718055994530942f;
      float f = 1.0f / l;
      if (a.head_sink && valid) f /= 1.0f + expf(a.head_sink[hq] - lse);
      if (valid && a.lse_out) a.lse_out[row] = lse;
      // The lanes of a quad hold 64 bytes of four rows each; transposed, a quad
      // stores 64 bytes of one row at a time (a thread's own 16-byte pieces of
      // 32 rows took the store path 4 times as long).
      const unsigned long long dst = valid ? reinterpret_cast<unsigned long long>(a.out + row * D) : 0;
      unsigned long long at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, dst, (lane & ~3) | i);
      __nv_bfloat162 sum = __floats2bfloat162_rn(0.0f, 0.0f);  // not finite if a result is not
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        dev::tmem_ld_cols<32>(o_col + c0, o);
        uint32_t x[4][4];  // [16-byte piece][word]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[2 * i] * f, o[2 * i + 1] * f);
          x[i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        {
          auto pair = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&x[i / 4][i % 4]); };
          __nv_bfloat162 t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = __hfma2(pair(i), pair(4 + i), __hmul2(pair(8 + i), pair(12 + i)));
          sum = __hadd2(sum, __hadd2(__hadd2(t[0], t[1]), __hadd2(t[2], t[3])));
        }
        dev::quad_transpose(x);
        // piece k is now this lane's 16 bytes of the quad's row k
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at[k])
            *reinterpret_cast<uint4*>(at[k] + 2 * c0 + 16 * (lane & 3)) = make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
      }
      const float2 s2 = __bfloat1622float2(sum);
      if (valid && !(fabsf(s2.x + s2.y) < INFINITY) && !care) spoilt[(un - 1) & 7] = un;
      if (care) {
        // the elements of V that were set to 0, to the rows that see them
        __syncwarp();
        const Range whole = whole_range(u, unit_tiles * tpt, W);
        for (int key = max(0, begin); valid && key <= pos; ++key) {
          if (key / kKeys >= whole.a && key / kKeys < whole.b) key = whole.b * kKeys;
          if (key > pos) break;
          const uint16_t* src = a.v + (size_t)(u.row0 + key) * a.v_stride + (size_t)u.head * D;
          for (int c = 0; c < D; ++c)
            if ((src[c] & 0x7F80u) == 0x7F80u) {
              __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out) + row * D + c;
              *o = __float2bfloat16(__bfloat162float(*o) + __uint_as_float((uint32_t)src[c] << 16));
            }
        }
      }
      ptx::tc_fence_before();
    }
  } else {
    if constexpr (kShares) ptx::regs_down<88>();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D, bool CAP>
cudaError_t launch_prompt(const CUtensorMap* tm, const PromptArgs& a, int sms, cudaStream_t stream) {
  using C = PromptCfg<D>;
  static std::atomic<int> smem_set[64];
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prompt_kernel<D, CAP>), smem_set, C::SMEM)) return e;
  const int tpt = 128 / a.group;
  // at most this many units of n tiles
  auto units = [&](int n) { return ((long long)a.total_tokens / (n * tpt) + a.batch) * a.num_kv_heads; };
  const int tiles = C::NQ > 1 && units(C::NQ) > sms ? C::NQ : 1;
  const long long most = units(tiles);
  const bool planned = most > sms || a.batch > kSmallBatch;
  const int grid = (int)(most < sms ? most : sms);
  if (planned) {
    const int threads = (a.batch + 31) / 32 * 32;
    if (cudaError_t e = launch_pdl(prompt_plan_kernel, 1, threads, 0, stream, a, tiles * tpt, grid)) return e;
  }
  return launch_pdl(prompt_kernel<D, CAP>, grid, C::THREADS, C::SMEM, stream, tm[0], tm[1], tm[2], a, tiles, planned);
}

}  // namespace

cudaError_t launch_attend_prompt(const CUtensorMap* tm, const PromptArgs& a, int sms, cudaStream_t stream) {
  const bool cap = a.softcap > 0.0f;
  switch (a.head_dim) {
    case 64: return cap ? launch_prompt<64, true>(tm, a, sms, stream) : launch_prompt<64, false>(tm, a, sms, stream);
    case 128: return cap ? launch_prompt<128, true>(tm, a, sms, stream) : launch_prompt<128, false>(tm, a, sms, stream);
    default: return cap ? launch_prompt<256, true>(tm, a, sms, stream) : launch_prompt<256, false>(tm, a, sms, stream);
  }
}

}  // namespace kvq
