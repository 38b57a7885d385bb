// tree_tile.cuh -- attention of many drafted nodes per kv head over the
// quantized paged cache on the tcgen05 tensor cores: kvq_attend_tree from 17
// query rows on (9 over long caches) at head_dim 128 and 256.
//
// Mathematics: for the row of a node, S_j = sm_scale <q, k_j> (capped) over the
// prefix keys j (of its window), its ancestors and itself; with a running
// reference mu and P_j = 2^(S_j log2 e - mu): o = sum P_j v_j / sum P_j, lse =
// ln 2 (mu + log2 sum P_j).
//
// A work unit is one (sequence, kv head) of up to 128 query rows, row r =
// node t * G + head g of the GQA group, with the split plan, producer, 64-key
// code stages and partial format of decode.cuh:
//
//   S [128 rows x 64 keys] = Q [128 x D] . K [64 x D]^T    A = Q in TMEM, B = K (f16, shared, K-major)
//   O [128 rows x D]    (+)= P [128 x 64] . V [64 x D]      A = P in TMEM, B = V (f16, shared, MN-major)
//
// Each key tile's codes are dequantized once into f16 tiles in shared memory
// (two of each), exactly: per-row scales go into the scores (K) and, under a
// power-of-two normaliser 2^F, into the weights (V), per-channel ones into Q
// and the output.  F is dev::ScaleUnit's: a node takes nothing of the precision
// of those that do not see it.  P overwrites its own S: head_dim 256 has two S
// buffers (Q 128 + O 256 + S 2 x 64 columns), head_dim 128 four.  One warp
// issues both products; their order in the tensor pipe is what keeps S, P and Q
// apart.
//
// Warp roles (20 warps, 18 and 19 for the even share of registers): 0-7 softmax
// (S -> P with lazy row maxima, 32 keys a thread; together Q of a piece into
// TMEM and the epilogue, half of the channels each); 8-11 K dequant, key
// 32 (w & 1) + lane, channel half w >> 1; 12-15 V dequant, the same; 16 TMA
// producer of the code stages; 17 the MMAs.
//
// A tile's softmax is a chain of latencies (tensor memory, row maximum,
// reference, weights) longer than its work, so a row's 64 keys go to two
// threads.  Rows past 64: warps 0-3 and 4-7 take the halves of the keys of every
// tile and agree on its maximum.  Up to 64 rows (FOLD): warps 0-3 take the even
// tiles and 4-7 the odd ones, and the halves are two copies of the row; the
// groups share O and with it a row's reference, which goes from tile to tile
// through shared memory; each keeps its own sum, under the reference it last saw.
//
// Bound: cache bytes for few rows of 8-bit codes, else the chain of a tile
// (conversion, QK^T, softmax, PV) and instruction issue, 0.45 of the slots.
// 131,072 int8 keys of head_dim 256, 16 nodes of 6 heads: 93 us, 2.9 TB/s; 4 x
// 32,768 int4 keys, 32 nodes: 276 us; 16 sequences to 32,768 fp8 keys, capped,
// 13 nodes of 4 heads: 246 us, 2.8 TB/s.
#pragma once

#include <type_traits>

#include "decode_tc.cuh"

namespace kvq {

namespace dev {

// Address of 16-byte f16 chunk c of key row kk in an f16 tile: 64-element slabs
// of [kTile rows][128 B] in the tensor core's 128-byte swizzle.
template <int SLAB>
__device__ __forceinline__ uint32_t tt_chunk(uint32_t tile, int kk, int c) {
  return tile + (uint32_t)(c >> 3) * SLAB + (uint32_t)kk * 128u + ((((uint32_t)c & 7u) ^ ((uint32_t)kk & 7u)) << 4);
}

}  // namespace dev

// SPLIT: the Q operand in two f16 parts (a per-channel K scale and an lse that
// is asked for).  At head_dim 128 the second part has tensor-memory columns of
// its own and a second pass of QK^T adds into the same S; at head_dim 256 a
// unit then has at most 64 rows, the second parts are the operand's rows
// 64..127, and warps 2 and 3 hand their rows of S to warps 0 and 1 through
// shared memory (as f16: 2^-11 of a 2^-12 correction).
// FOLD (not with that): units of at most 64 rows stand in the tile twice, and
// each copy takes 32 keys of every tile as a row of its own (P is 0 at the
// others), so that all four warps of a group have half a tile's softmax each;
// the epilogue adds the copies up.
// CAP: a softcap.
template <int DT, int D, bool SPLIT, bool CAP, bool FOLD>
__global__ void __launch_bounds__(kTtWarps * 32, 1)
    tree_tile_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const DecodeArgs a) {
  using Gm = Geo<DT, D, kTile>;
  constexpr bool STACK = SPLIT && D == 256;
  constexpr int KT = kTile, SLAB = KT * 128, TILE = (D / 64) * SLAB;
  // TMEM columns
  constexpr int Q_COL = 0, QL_COL = D / 2, O_COL = D / 2 * (SPLIT && !STACK ? 2 : 1), S_COL = O_COL + D;
  static_assert(S_COL + 2 * KT <= 512, "TMEM columns");
  using Order = TileOrder<KT, true>;
  constexpr int kDqK = 8, kDqV = 12, kProducer = 16, kMma = 17;
  constexpr int NSB = S_COL + 4 * KT <= 512 ? 4 : 2;  // S buffers
  constexpr int LA = NSB - 1;                          // tiles of QK^T ahead of PV
  constexpr int CH = KT / 2;                           // keys of a softmax thread in a tile
  static_assert(!(FOLD && STACK), "one use of the second 64 rows");
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const TtSmem lay = tt_smem_layout(D, a.stages, a.batch, a.stage_stride, tt_exchange(D, SPLIT, FOLD));
  uint8_t* ring = base + lay.ring;
  const uint32_t kf = ptx::smem_u32(base + lay.kf), vf = ptx::smem_u32(base + lay.vf);
  float* ksb = reinterpret_cast<float*>(base + lay.sc);  // [8][KT] K scales of tile it, at it & 7
  float* vsb = ksb + 8 * KT;                              // [8][KT] its V scales over 2^F
  // [8] F, how far it has grown since the tile before, how far the scales (of the
  // tile; where all rows see them, of those so far) are above 2^F
  float4* funit = reinterpret_cast<float4*>(vsb + 8 * KT);
  float* ref = reinterpret_cast<float*>(base + lay.pair);  // [128] the rows' reference maxima
  float* part = ref + kTtRows;                             // [2][2 groups][128] a tile's maxima; last references and sums
  int* pl_pre = reinterpret_cast<int*>(base + lay.pre);
  int* pl_misc = pl_pre + a.batch + 1;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(base + lay.bars);
  uint64_t* bar_empty = bar_full + a.stages;
  uint64_t* b_s = bar_empty + a.stages;  // [NSB] QK^T of tile it complete: S buffer it % NSB, K tile it & 1
  uint64_t* b_pv = b_s + 4;              // [NSB] PV of tile it complete: V tile it & 1 free
  uint64_t* b_kfull = b_s + 8;           // [2] K f16 tile written
  uint64_t* b_vfull = b_s + 10;          // [2] V f16 tile written
  uint64_t* b_p = b_s + 12;              // [NSB] P of tile it written (and O rescaled)
  uint64_t* b_q = b_s + 16;              // Q of a piece in TMEM
  uint64_t* b_ksc = b_s + 17;            // [8] K scales of tile it (per-row K)
  uint64_t* b_vsc = b_s + 25;            // [8] V scales of tile it (per-row V)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + lay.slot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&bar_full[s], 1);
      ptx::mbar_init(&bar_empty[s], 8);  // K and V dequant warps
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&b_kfull[i], 4);
      ptx::mbar_init(&b_vfull[i], 4);
    }
    ptx::mbar_init(b_q, 8);
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&b_s[i], 1);
      ptx::mbar_init(&b_pv[i], 1);
      ptx::mbar_init(&b_p[i], FOLD ? 4 : 8);  // the softmax warps of a tile
    }
    for (int i = 0; i < 8; ++i) {
      ptx::mbar_init(&b_ksc[i], 2);
      ptx::mbar_init(&b_vsc[i], 2);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMma) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  const Slice<KT, true> sp = build_slice<KT, true>(a, pl_pre, pl_misc);
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Bounded wait: after a timeout every later wait of the CTA is skipped, the
  // results are flagged, and the CTA reaches its end.  (No calls in this kernel:
  // with them the warpgroups' register shares would not hold.)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ptx::mbar_try_wait(bar, parity) || *abort_flag) return;
    if (!ptx::mbar_wait_bounded_inl(bar, parity)) {
      *abort_flag = 1;
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    }
  };
  const bool k_row = a.k_mode == KVQ_SCALE_PER_ROW, v_row = a.v_mode == KVQ_SCALE_PER_ROW;

  if (warp >= kProducer) ptx::regs_down<64>();
  if (warp == kProducer) {
    // ============================================================ producer
    produce_lanes<Gm, true, true>(a, sp, &tmk, &tmv, ring, bar_full, bar_empty, pl_pre, pl_misc);
  } else if (warp >= kDqK && warp < kDqV + 4) {
    // ==================================================== K and V dequant
    // A stage's codes are read at once and converted 64 of a row at a time; the
    // wait for the MMA that frees the f16 tile comes before the first store.
    ptx::regs_down<88>();
    const bool is_v = warp >= kDqV;
    const int q = warp - (is_v ? kDqV : kDqK);
    const int kk = 32 * (q & 1) + lane, hf = q >> 1;
    constexpr int HB = Gm::DP / 2;                // code bytes of a channel half
    constexpr int PB = DT == KVQ_INT4 ? 32 : 64;  // of a piece
    constexpr int PC = PB / 16;                   // its 16-byte chunks
    constexpr int CW = DT == KVQ_INT4 ? 16 : 8;   // f16 pairs of a chunk
    uint64_t* b_free = is_v ? b_pv : b_s;
    uint64_t* b_full = is_v ? b_vfull : b_kfull;
    const uint32_t f16_base = is_v ? vf : kf;
    const uint32_t code_off = is_v ? (uint32_t)Gm::CODE_BYTES : 0u;
    const bool scaled = (is_v ? v_row : k_row) && hf == 0;
    uint32_t it = 0;
    RingPos rp;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      dev::ScaleUnit unit;  // of the piece's V scales
      int F_last = 0;
      const VSeq vs = a.vseq[b];
      const int first_key = vs.lo;  // (a row below it may hold anything)
      const int c_lo = vs.gaps, c_hi = a.key_end[vs.tok0];  // the keys that all rows see
      for (int key0 = Order::first(k0, k1); Order::more(key0, k0, k1); key0 += Order::step, ++it, rp.next(a.stages)) {
        wait(&bar_full[rp.stage], rp.phase);
        const uint8_t* st = ring + (size_t)rp.stage * a.stage_stride;
        if (scaled) {
          // Slot it & 7 was last read by the softmax of it - 8.  K: this warp has
          // waited for QK^T of it - 3, issued after PV of it - 3 - NSB, whose softmax
          // was done; V: for PV of it - 3.
          const float* scp = reinterpret_cast<const float*>(st + 2 * Gm::CODE_BYTES + (is_v ? KT * 4 : 0));
          float sc = scp[kk];
          if (is_v) {
            auto seen = [&](int key) { return key >= first_key && key < L; };
            float vm = seen(key0 + lane) ? dev::finite_or_0(scp[lane]) : 0.0f;
            if (seen(key0 + 32 + lane)) vm = fmaxf(vm, dev::finite_or_0(scp[32 + lane]));
            vm = ptx::redux_max(vm);
            const bool common = key0 >= c_lo && key0 + KT <= c_hi;
            const int f = dev::scale_exponent(vm), F = unit.next(f, common);
            vsb[(it & 7) * KT + kk] = seen(key0 + kk) ? sc * dev::pow2i(-F) : 0.0f;
            if (q == 0 && lane == 0) {
              const bool first = key0 == Order::first(k0, k1);
              funit[it & 7] = make_float4(__int_as_float(F), first ? 0.0f : (float)min(F - F_last, dev::ScaleUnit::kMost),
                                          (float)((common ? unit.all : f) - F), 0.0f);
            }
            F_last = F;
          } else {
            ksb[(it & 7) * KT + kk] = sc;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(is_v ? &b_vsc[it & 7] : &b_ksc[it & 7]);
        }
        const uint32_t buf = it & 1, tile = f16_base + buf * TILE;
        // (all of the codes first: the sooner the stage is free, the more of the
        // cache is on its way)
        uint4 w[HB / 16];
#pragma unroll
        for (int j = 0; j < HB / 16; ++j) {
          const uint32_t byte = (uint32_t)(hf * HB + 16 * j);
          w[j] = *reinterpret_cast<const uint4*>(st + code_off + (byte / Gm::SPAN) * (KT * Gm::SPAN) +
                                                 dev::swz<Gm::SPAN>((uint32_t)kk * Gm::SPAN + byte % Gm::SPAN));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar_empty[rp.stage]);
#pragma unroll
        for (int pc = 0; pc < HB / PB; ++pc) {
          uint32_t v[PC * CW];
#pragma unroll
          for (int j = 0; j < PC; ++j) dev::k_cols<DT>(w[pc * PC + j], v + CW * j);
          if (DT == KVQ_FP8_E4M3 && is_v) {  // (a key no row sees may hold NaN codes: they lose against -448)
#pragma unroll
            for (int j = 0; j < PC * CW; ++j) v[j] = ptx::max_f16x2(v[j], 0xDF00DF00u);
          }
          // the MMA two tiles back has read this f16 tile
          if (pc == 0 && it >= 2) wait(&b_free[(it - 2) % NSB], ((it - 2) / NSB) & 1);
#pragma unroll
          for (int c = 0; c < PC * CW / 4; ++c) {
            const uint32_t addr = dev::tt_chunk<SLAB>(tile, kk, hf * (D / 16) + pc * (PC * CW / 4) + c);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[4 * c]), "r"(v[4 * c + 1]),
                         "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                         : "memory");
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b_full[buf]);
      }
    }
  } else if (warp == kMma) {
    // ================================================================ MMA
    // QK^T(it + LA), PV(it), QK^T(it + LA + 1), ...: executed in this order, and
    // LA < NSB, so an S buffer is written again after PV has read its P there.
    constexpr uint32_t idesc_qk = ptx::idesc_f16_f32(128, KT);
    constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, D) | (1u << 16);  // B MN-major
    const uint64_t kd = ptx::smem_desc_sw128(kf);
    const uint32_t k_lo = (uint32_t)kd, d_hi = (uint32_t)(kd >> 32);
    const uint32_t v_lo = (uint32_t)ptx::smem_desc_sw128_mn(vf, SLAB);
    auto issue_qk = [&](uint32_t j) {
      const uint32_t buf = j & 1, s_col = tmem + S_COL + KT * (j % NSB);
      wait(&b_kfull[buf], (j >> 1) & 1);
      __syncwarp();
      ptx::tc_fence_after();
      if constexpr (SPLIT && !STACK) {
        // the small part first: less is rounded
#pragma unroll
        for (int sl = 0; sl < D / 64; ++sl)
          ptx::mma_f16_ts_x4(s_col, tmem + QL_COL + 32 * sl, 8, k_lo + ((buf * TILE + sl * SLAB) >> 4),
                             d_hi, idesc_qk, sl > 0 ? 1u : 0u);
      }
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl)
        ptx::mma_f16_ts_x4(s_col, tmem + Q_COL + 32 * sl, 8, k_lo + ((buf * TILE + sl * SLAB) >> 4),
                           d_hi, idesc_qk, sl > 0 || (SPLIT && !STACK) ? 1u : 0u);
      ptx::mma_commit(&b_s[j % NSB]);
    };
    // a piece's first PV overwrites O
    auto issue_pv = [&](uint32_t j, bool first) {
      const uint32_t buf = j & 1;
      wait(&b_vfull[buf], (j >> 1) & 1);
      wait(&b_p[j % NSB], (j / NSB) & 1);
      __syncwarp();
      ptx::tc_fence_after();
      ptx::mma_f16_ts_x4_step(tmem + O_COL, tmem + S_COL + KT * (j % NSB), 8, v_lo + buf * (TILE >> 4), (16 * 128) >> 4, d_hi,
                              idesc_pv, first ? 0u : 1u);
      ptx::mma_commit(&b_pv[j % NSB]);
    };
    uint32_t it = 0;
    int pc = 0;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next, ++pc) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      wait(b_q, pc & 1);
      const uint32_t n = (uint32_t)((k1 - k0 + KT - 1) / KT);
      for (uint32_t i = 0; i < n && i < LA; ++i) issue_qk(it + i);
      for (uint32_t i = 0; i < n; ++i, ++it) {
        if (i + LA < n) issue_qk(it + LA);
        issue_pv(it, i == 0);
      }
    }
    // every MMA has completed before TMEM can be released
    if (it > 0 && !ptx::mbar_wait_bounded_inl(&b_pv[(it - 1) % NSB], ((it - 1) / NSB) & 1) && lane == 0)
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    __syncwarp();
  } else if (warp < kDqK) {
    // ============================================================ softmax
    ptx::regs_up<120>();
    const int q = warp & 3, grp = warp >> 2;  // TMEM lane quarter; even or odd tiles
    // query row = TMEM lane (STACK: lanes 64..127 hold the second parts of rows 0..63,
    // FOLD: rows 0..63 again)
    const int r = STACK || FOLD ? (32 * q + lane) & 63 : 32 * q + lane;
    const bool second = STACK && q >= 2;
    const int part0 = CH * (FOLD ? q >> 1 : grp);  // first key of this thread in a tile
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16);
    const int G = a.group, Hq = a.num_q_heads, rows = a.rows;
    const uint32_t exch = ptx::smem_u32(base + lay.exch);
    // S of the second parts, [2 tiles][2 groups][64 rows][CH keys] f16, 16-byte chunks XOR (row >> 1 & 3)
    auto exch_at = [&](uint32_t it, int chunk) -> uint32_t {
      return exch + ((it & 1) * 2 + grp) * (64 * CH * 2) + (uint32_t)r * (CH * 2) + (((uint32_t)chunk ^ ((uint32_t)r >> 1 & 3u)) << 4);
    };
    const int bar_mine = 1 + q + 4 * grp, bar_other = 1 + q + 4 * (grp ^ 1);  // "the other group's reference is there"
    const int bar_exch = 9 + (q & 1) + 2 * grp;
    const int t_row = dev::div_small(r, __frcp_rn((float)G));
    uint32_t it = 0;
    int pc = 0;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next, ++pc) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      const VSeq vs = a.vseq[b];
      const bool valid = r < rows && t_row < vs.ntok;
      const bool idle = !__any_sync(0xffffffffu, valid);  // rows of no node: what they hold is read by nobody
      const size_t tok = (size_t)vs.tok0 + t_row;
      const int hq = h * G + (r - t_row * G);
      dev::RowRule ru{};
      bool blind = !valid;
      float alpha = 1.0f;
      // ---- Q of this piece (every QK^T of the previous one has completed: this
      // thread waited for its last PV): the per-channel K scale folded in under a
      // power-of-two normaliser, the row normalised by the power of two at or
      // above its maximum, f16 pairs in the K order of the K
      // tile (each of the row's two threads writes half of the channels).
      if (!idle) {
        const bool kc = a.k_mode == KVQ_SCALE_PER_CHANNEL;
        const uint16_t* src = a.q + (tok * Hq + hq) * D;
        const float* ksp = a.k_scale + (size_t)h * D;
        int ek = 0;
        if (kc) {
          float km = 0.0f;
#pragma unroll
          for (int c = 4 * lane; c < D; c += 128) {
            const float4 s4 = __ldg(reinterpret_cast<const float4*>(ksp + c));
            km = fmaxf(fmaxf(km, fmaxf(fabsf(s4.x), fabsf(s4.y))), fmaxf(fabsf(s4.z), fabsf(s4.w)));
          }
          km = ptx::redux_max(km);
          ek = km > 0.0f ? min(126, max(-126, dev::ceil_log2(km))) : 0;
        }
        const float sk = dev::pow2i(-ek);
        auto unpack = [&](const uint4 raw, int c8, float (&qv)[8]) {
          const uint32_t ww[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            qv[2 * j] = __uint_as_float(ww[j] << 16);
            qv[2 * j + 1] = __uint_as_float(ww[j] & 0xFFFF0000u);
          }
          if (kc) {
            const float4 s0 = __ldg(reinterpret_cast<const float4*>(ksp + 8 * c8));
            const float4 s1 = __ldg(reinterpret_cast<const float4*>(ksp + 8 * c8 + 4));
            qv[0] *= s0.x * sk; qv[1] *= s0.y * sk; qv[2] *= s0.z * sk; qv[3] *= s0.w * sk;
            qv[4] *= s1.x * sk; qv[5] *= s1.y * sk; qv[6] *= s1.z * sk; qv[7] *= s1.w * sk;
          }
        };
        constexpr int NCH8 = D / 8, BAT = 8;
        float qm = 0.0f;
#pragma unroll 1
        for (int c0 = 0; c0 < NCH8; c0 += BAT) {
          uint4 raw[BAT];
#pragma unroll
          for (int i = 0; i < BAT; ++i) raw[i] = valid ? ptx::ldg_nc_v4(src + 8 * (c0 + i)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < BAT; ++i) {
            float qv[8];
            unpack(raw[i], c0 + i, qv);
#pragma unroll
            for (int j = 0; j < 8; ++j) qm = fmaxf(qm, fabsf(qv[j]));
          }
        }
        const int eq = qm > 0.0f ? min(126, max(-126, dev::ceil_log2(qm))) : 0;
        const float sq = dev::pow2i(-eq);
#pragma unroll 1
        for (int c32 = grp * (D / 64); c32 < (grp + 1) * (D / 64); ++c32) {
          uint4 raw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[i] = valid ? ptx::ldg_nc_v4(src + 8 * (4 * c32 + i)) : make_uint4(0, 0, 0, 0);
          uint32_t w[16], lo[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float qv[8];
            unpack(raw[i], 4 * c32 + i, qv);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float f = DT == KVQ_INT4 && (m & 1) ? sq * dev::odd_channel_factor<DT>() : sq;  // (channels m, m + 4)
              const float q0 = DT == KVQ_INT4 ? qv[m] : qv[2 * m], q1 = DT == KVQ_INT4 ? qv[m + 4] : qv[2 * m + 1];
              w[4 * i + m] = dev::pack_h2(q0 * f, q1 * f);
              if constexpr (SPLIT) lo[4 * i + m] = dev::rest_h2(q0 * f, q1 * f, w[4 * i + m]);
            }
          }
          if constexpr (STACK) {
            if (second) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = lo[i];
            }
          } else if constexpr (SPLIT) {
            ptx::tmem_st16(t_lane + QL_COL + 16 * c32, lo);
          }
          ptx::tmem_st16(t_lane + Q_COL + 16 * c32, w);
        }
        ptx::tmem_wait_st();
        float base_f = a.sm_scale;
        if (a.k_mode == KVQ_SCALE_PER_TENSOR) base_f *= a.k_scale[0];
        base_f *= CAP ? 1.0f / a.softcap : kLog2e;
        // base * 2^(ek + eq) in two exact power-of-two steps, finite and > 0 (so
        // that alpha * -inf stays -inf)
        const int e = ek + eq, e1 = e / 2;
        alpha = valid ? fmaxf(fminf(base_f * dev::pow2i(e1) * dev::pow2i(e - e1), 3.4028234e38f), 1.17549435e-38f) : 1.0f;
        // Rows that see none of the piece's keys (of no node, or all of them
        // outside a window) are scored like any other and count for nothing
        // at the end: hiding every key of every tile would take longer.
        ru.end = L;
        ru.bits = -1;
        if (valid) {
          const dev::RowRule rr = dev::row_rule<true>(a, tok, vs.pos0 + t_row, hq, L);
          blind = rr.begin == 0x7FFFFFFF || (max(rr.begin, k0) >= min(rr.end, k1) && k1 <= rr.end);
          if (!blind) ru = rr;
        }
        ptx::tc_fence_before();
        __syncwarp();
      }
      if (lane == 0) ptx::mbar_arrive(b_q);

      const float cap2 = CAP ? a.softcap * kLog2e : 0.0f;
      const ptx::f32x2 aa = ptx::pack_x2(alpha, alpha);

      float mu = -INFINITY;                      // this row's reference (log2 units) as of this group's last tile
      ptx::f32x2 l2 = ptx::pack_x2(0.0f, 0.0f), l3 = l2;  // its weight sum there, in four parts
      for (int key0 = Order::first(k0, k1); Order::more(key0, k0, k1); key0 += Order::step, ++it) {
        if (FOLD && (int)(it & 1) != grp) continue;
        const bool first = key0 == Order::first(k0, k1), last = !Order::more(key0 + Order::step, k0, k1);
        const uint32_t s_col = t_lane + S_COL + KT * (it % NSB);
        wait(&b_s[it % NSB], (it / NSB) & 1);
        if (idle) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&b_p[it % NSB]);
          continue;
        }
        ptx::tc_fence_after();
        if constexpr (STACK) {
          // (a place is written again two tiles on, past the barrier of the tile between)
          if (second) {
            float y[CH];
            dev::tmem_ld_cols<CH>(s_col + part0, y);
#pragma unroll
            for (int c8 = 0; c8 < CH / 8; ++c8)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(exch_at(it, c8)),
                           "r"(dev::pack_h2(y[8 * c8], y[8 * c8 + 1])), "r"(dev::pack_h2(y[8 * c8 + 2], y[8 * c8 + 3])),
                           "r"(dev::pack_h2(y[8 * c8 + 4], y[8 * c8 + 5])), "r"(dev::pack_h2(y[8 * c8 + 6], y[8 * c8 + 7]))
                           : "memory");
            __syncwarp();
            ptx::named_bar_sync(bar_exch, 64);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&b_p[it % NSB]);
            continue;
          }
        }
        if (k_row) wait(&b_ksc[it & 7], (it >> 3) & 1);
        const float* ksc = ksb + (it & 7) * KT;
        const float* vsc = vsb + (it & 7) * KT;
        const bool full = key0 >= ru.begin && key0 + KT <= ru.end;
        uint32_t bits[2] = {0u, 0u};  // visible keys of a tile that is not whole
        float lift = 0.0f;            // how far the V scales that the row sees of it are above 2^F
        if (!full) {
          if (key0 + KT > ru.end) dev::tree_sees_64(a, ru, key0, bits);
          const int lo = min(KT, max(0, ru.begin - key0)), hi = min(KT, max(0, ru.end - key0));
          if (lo < hi) {
            const uint64_t in = (hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((1ull << lo) - 1);
            bits[0] |= (uint32_t)in;
            bits[1] |= (uint32_t)(in >> 32);
          }
          if (v_row) {
            // (a row's two threads find the same; FOLD: each copy for its own keys)
            wait(&b_vsc[it & 7], (it >> 3) & 1);
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < KT; k += 4) {
              if (FOLD && (k < 32) != (part0 == 0)) continue;
              const float4 s4 = *reinterpret_cast<const float4*>(vsc + k);
              const uint32_t b4 = (k < 32 ? bits[0] : bits[1]) >> (k & 31);
              top = fmaxf(top, fmaxf(fmaxf(b4 & 1u ? dev::finite_or_0(s4.x) : 0.0f, b4 & 2u ? dev::finite_or_0(s4.y) : 0.0f),
                                     fmaxf(b4 & 4u ? dev::finite_or_0(s4.z) : 0.0f, b4 & 8u ? dev::finite_or_0(s4.w) : 0.0f)));
            }
            lift = dev::scale_lift(top, 0);
          }
          if (part0) bits[0] = bits[1];
        }
        // scores, with a per-row K scale (and 1 / softcap) in
        float y[CH];
        {
          uint32_t v[CH];
          ptx::tmem_ld32(s_col + part0, v);
          auto scores = [&]() {
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < CH; ++k) {
              asm volatile("" : "+r"(v[k]));
              y[k] = __uint_as_float(v[k]);
            }
          };
          if (!STACK && k_row) {
            float4 s4[CH / 4];  // (on their way before the scores are there)
#pragma unroll
            for (int k = 0; k < CH / 4; ++k) s4[k] = *reinterpret_cast<const float4*>(ksc + part0 + 4 * k);
            scores();
#pragma unroll
            for (int k = 0; k < CH; k += 4) {
              ptx::mul_x2(y[k], y[k + 1], y[k], y[k + 1], s4[k / 4].x, s4[k / 4].y);
              ptx::mul_x2(y[k + 2], y[k + 3], y[k + 2], y[k + 3], s4[k / 4].z, s4[k / 4].w);
            }
          } else {
            scores();
          }
          if constexpr (STACK) {
            __syncwarp();
            ptx::named_bar_sync(bar_exch, 64);
#pragma unroll
            for (int c8 = 0; c8 < CH / 8; ++c8) {
              uint32_t w[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                           : "r"(exch_at(it, c8))
                           : "memory");
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                y[8 * c8 + 2 * j] += f.x;
                y[8 * c8 + 2 * j + 1] += f.y;
              }
            }
          }
        }
        if constexpr (CAP) {
#pragma unroll
          for (int k = 0; k < CH; k += 2) ptx::mul_x2(y[k], y[k + 1], y[k], y[k + 1], alpha, alpha);
        }
        if (!full) {  // keys that this row does not see
#pragma unroll
          for (int k = 0; k < CH; ++k)
            if (!((bits[0] >> k) & 1u)) y[k] = -INFINITY;
        }
        float m, least = INFINITY;
        {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mn[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
          for (int k = 0; k < CH; k += 2) {
            mx[k / 2 % 4] = ptx::max3(mx[k / 2 % 4], y[k], y[k + 1]);
            if constexpr (CAP) mn[k / 2 % 4] = ptx::min3(mn[k / 2 % 4], y[k], y[k + 1]);
          }
          m = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
          if constexpr (CAP) least = fminf(ptx::min3(mn[0], mn[1], mn[2]), mn[3]);
        }
        // (rows that count for nothing may hold anything)
        const bool near = CAP && __all_sync(0xffffffffu, blind || fmaxf(fabsf(m), fabsf(least)) <= dev::CapNear::kReach);
        if constexpr (!FOLD) {
          // the row's other half (a place is written again two tiles on, past the
          // barrier of the tile between); both have S in registers before either
          // writes its part of P over it
          float* place = part + 256 * (it & 1) + 32 * q + lane;
          place[128 * grp] = m;
          ptx::tc_fence_before();
          __syncwarp();
          ptx::named_bar_sync(1 + q, 64);
          ptx::tc_fence_after();
          m = fmaxf(m, place[128 * (grp ^ 1)]);
        }
        if constexpr (CAP) {
          if (fabsf(m) <= dev::CapNear::kReach) {
            m = dev::CapNear(cap2, 1.0f).score(m);
          } else if (m != -INFINITY) {
            float x[2] = {m, 0.0f};
            dev::cap_scores<2>(x, cap2);
            m = x[0];
          }
        } else {
          m *= alpha;
        }
        float grown = 0.0f;  // F since the last tile
        if (v_row) {
          wait(&b_vsc[it & 7], (it >> 3) & 1);
          const float4 fu = funit[it & 7];
          m += full ? fu.z : lift;
          grown = fu.y;
        }
        // The reference (FOLD: that the other group left at the tile before) moves
        // only when this tile's maximum exceeds it by more than 8 (P <= 2^8 in
        // f16), and against F, which leaves O as it is; a row with no key yet holds
        // zeros in O.
        float was = mu;
        if (FOLD && !first) {
          __syncwarp();
          ptx::named_bar_sync(bar_mine, 64);
          was = ref[32 * q + lane];
        }
        was -= grown;
        const float now = m > was + 8.0f ? m : was;
        if (FOLD && !last) {
          ref[32 * q + lane] = now;
          __syncwarp();
          ptx::named_bar_arrive(bar_other, 64);
        }
        const float corr = now != was && was != -INFINITY ? ptx::fast_exp2(was - now) : 1.0f;
        if (now != mu) {
          const float c = mu != -INFINITY ? ptx::fast_exp2(mu - now) : 1.0f;
          l2 = ptx::mul_x2(l2, ptx::pack_x2(c, c));
          l3 = ptx::mul_x2(l3, ptx::pack_x2(c, c));
          mu = now;
        }
        if (__any_sync(0xffffffffu, !first && corr != 1.0f)) {
          // bring O (a row's two threads half of the channels each, FOLD: all) to the
          // new reference, after the previous PV has landed
          wait(&b_pv[(it - 1) % NSB], ((it - 1) / NSB) & 1);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c0 = FOLD ? 0 : grp * (D / 2); c0 < (FOLD ? D : (grp + 1) * (D / 2)); c0 += 16) {
            float o[16];
            dev::tmem_ld_cols<16>(t_lane + O_COL + c0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= corr;
            dev::tmem_st_cols<16>(t_lane + O_COL + c0, o);
          }
        }
        // P = 2^(y - mu), with the V scales, f16 pairs; the sums take the fp32
        // weights
        const float nmu = mu == -INFINITY ? 0.0f : -mu;
        const ptx::f32x2 nm = ptx::pack_x2(nmu, nmu);
        if constexpr (FOLD) {
          const uint32_t none[16] = {};
          __syncwarp();
          ptx::tmem_st16(s_col + (CH - part0) / 2, none);
        }
        // rows: per-row V scales, some: of a tile that is not whole (the scales of
        // hidden keys may be anything)
        auto weigh_as = [&](auto&& score, auto rows, auto some) {
          constexpr bool VR = decltype(rows)::value, SOME = decltype(some)::value;
          uint32_t p[CH / 2];
#pragma unroll
          for (int k = 0; k < CH; k += 4) {
            float4 s4;
            if constexpr (VR) s4 = *reinterpret_cast<const float4*>(vsc + part0 + k);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float z0, z1;
              ptx::unpack_x2(score(ptx::pack_x2(y[k + 2 * j], y[k + 2 * j + 1])), z0, z1);
              const ptx::f32x2 e = ptx::pack_x2(ptx::fast_exp2(z0), ptx::fast_exp2(z1));
              if (j) l3 = ptx::add_x2(l3, e);
              else l2 = ptx::add_x2(l2, e);
              float e0, e1;
              ptx::unpack_x2(e, e0, e1);
              if constexpr (SOME) {
                e0 = dev::scaled<true>(e0, j ? s4.z : s4.x);
                e1 = dev::scaled<true>(e1, j ? s4.w : s4.y);
              } else if constexpr (VR) {
                ptx::mul_x2(e0, e1, e0, e1, j ? s4.z : s4.x, j ? s4.w : s4.y);
              }
              p[k / 2 + j] = dev::pack_h2(e0, e1);
            }
          }
          __syncwarp();
          ptx::tmem_st16(s_col + part0 / 2, p);
        };
        // (one branch here, the same for a warp: one at each key would keep the keys apart)
        const bool whole_tile = __all_sync(0xffffffffu, full);
        auto weigh = [&](auto&& score) {
          if (!v_row) weigh_as(score, std::false_type{}, std::false_type{});
          else if (whole_tile) weigh_as(score, std::true_type{}, std::false_type{});
          else weigh_as(score, std::true_type{}, std::true_type{});
        };
        if constexpr (!CAP) {
          weigh([&](ptx::f32x2 x) { return ptx::fma_x2(x, aa, nm); });
        } else if (near) {
          // (of a tile with hidden keys, of score -inf, not all rows are near)
          const dev::CapNear cap_near(cap2, 1.0f);
          weigh([&](ptx::f32x2 x) { return cap_near.scores(x, nm); });
        } else {
#pragma unroll
          for (int c = 0; c < CH; c += 16) {
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = y[c + k];
            dev::cap_scores<16>(x, cap2);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (y[c + k] != -INFINITY) y[c + k] = x[k];  // (a hidden key stays -inf)
          }
          weigh([&](ptx::f32x2 x) { return ptx::add_x2(x, nm); });
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b_p[it % NSB]);
      }

      // ---- epilogue: O out of TMEM, normalised.  The workspace and the output
      // are written after the preceding grid (the producer waited for it before
      // the first tile's codes).  A unit of one piece (`whole`) is finished here:
      // head sink, static V scale and bf16, as in the combine; otherwise the
      // partial with its base-2 log-sum-exp.
      if (it > 1) wait(&b_pv[(it - 2) % NSB], ((it - 2) / NSB) & 1);
      wait(&b_pv[(it - 1) % NSB], ((it - 1) / NSB) & 1);
      if (idle || second) continue;
      ptx::tc_fence_after();
      // both groups' sums under the last reference (FOLD: the last tile's group has it)
      float l, mu_o;
      {
        float lb;
        ptx::unpack_x2(ptx::add_x2(l2, l3), l, lb);
        l += lb;
        part[256 * grp + 32 * q + lane] = mu;
        part[256 * grp + 128 + 32 * q + lane] = l;
        __syncwarp();
        ptx::named_bar_sync(1 + q, 64);
        mu_o = part[256 * (grp ^ 1) + 32 * q + lane];
        lb = part[256 * (grp ^ 1) + 128 + 32 * q + lane];
        const float top = !FOLD || (int)((it - 1) & 1) == grp ? mu : mu_o;
        if (mu != top) l *= ptx::fast_exp2(mu - top);
        if (mu_o != top) lb *= ptx::fast_exp2(mu_o - top);
        mu = top;
        l = blind ? 0.0f : l + lb;
      }
      // FOLD: both copies of a row under one reference; the second sends its O,
      // 16 columns at a time (a place is written again two steps on, past the
      // barrier of the step between)
      float copy = 1.0f;
      float* fold = reinterpret_cast<float*>(base + lay.exch);
      float4* fold_o = reinterpret_cast<float4*>(fold + 512) + (2 * grp + (q & 1)) * 256;  // [2 steps][4][32 rows]
      if constexpr (FOLD) {
        float* f = fold + 256 * grp + 32 * q + lane;
        f[0] = mu;
        f[128] = l;
        __syncwarp();
        ptx::named_bar_sync(bar_exch, 64);
        f = fold + 256 * grp + 32 * (q ^ 2) + lane;
        const float top = fmaxf(mu, f[0]);
        if (mu != top) copy = ptx::fast_exp2(mu - top);
        l = l * copy + f[128] * (f[0] != top ? ptx::fast_exp2(f[0] - top) : 1.0f);
        mu = top;
        if (q >= 2) {
          if (l == 0.0f) copy = 0.0f;
#pragma unroll 1
          for (int c0 = grp * (D / 2); c0 < (grp + 1) * (D / 2); c0 += 16) {
            float o[16];
            dev::tmem_ld_cols<16>(t_lane + O_COL + c0, o);
            float4* to = fold_o + (c0 / 16 & 1) * 128 + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              to[32 * j] = make_float4(o[4 * j] * copy, o[4 * j + 1] * copy, o[4 * j + 2] * copy, o[4 * j + 3] * copy);
            __syncwarp();
            ptx::named_bar_sync(bar_exch, 64);
          }
          ptx::tc_fence_before();
          continue;
        }
      }
      const int F = v_row ? __float_as_int(funit[(it - 1) & 7].x) : 0;
      const bool some = l != 0.0f;  // (or NaN)
      float inv = some ? (v_row ? dev::pow2i(F) : 1.0f) / l : 0.0f;
      const bool whole = k0 == (vs.lo & ~(KT - 1)) && k1 == L;
      // channels c0 .. c0 + 15 of this thread's row, in channel order
      auto channels = [&](int c0, float (&x)[16]) {
        float o[16];
        dev::tmem_ld_cols<16>(t_lane + O_COL + c0, o);
        if constexpr (FOLD) {
          __syncwarp();
          ptx::named_bar_sync(bar_exch, 64);
          const float4* from = fold_o + (c0 / 16 & 1) * 128 + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 x4 = from[32 * j];
            o[4 * j] = o[4 * j] * copy + x4.x;
            o[4 * j + 1] = o[4 * j + 1] * copy + x4.y;
            o[4 * j + 2] = o[4 * j + 2] * copy + x4.z;
            o[4 * j + 3] = o[4 * j + 3] * copy + x4.w;
          }
        }
        if (!some) {  // (O may hold anything)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        }
        if constexpr (DT == KVQ_INT4) {
          // N index 8 i + 2 m + e holds channel 8 i + m + 4 e, odd m times 16
#pragma unroll
          for (int g8 = 0; g8 < 2; ++g8)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float cf = (m & 1) ? dev::odd_channel_factor<DT>() : 1.0f;
              x[8 * g8 + m] = o[8 * g8 + 2 * m] * inv * cf;
              x[8 * g8 + m + 4] = o[8 * g8 + 2 * m + 1] * inv * cf;
            }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = o[i] * inv;
        }
      };
      unsigned long long dst;
      if (whole) {
        float lse = -INFINITY;
        if (some) {
          lse = (mu + ptx::fast_log2(l)) * 0.69314718055994530942f;
          if (a.head_sink && valid) inv /= 1.0f + expf(a.head_sink[hq] - lse);
        }
        if (a.v_mode == KVQ_SCALE_PER_TENSOR) inv *= a.v_scale[0];
        if (valid && grp == 0 && a.lse_out) a.lse_out[tok * Hq + hq] = lse;
        dst = reinterpret_cast<unsigned long long>(a.out + (tok * Hq + hq) * a.out_dim);
      } else {
        if (valid && grp == 0) a.part_lse[(size_t)u * rows + r] = dev::part_lse<true>(mu, l);
        dst = reinterpret_cast<unsigned long long>(a.part_o + ((size_t)u * rows + r) * D);
      }
      // quads of lanes store 64 bytes of a row at a time
      if (!valid) dst = 0;
      unsigned long long at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, dst, (lane & ~3) | i);
      const float* vs_ch = whole && a.v_mode == KVQ_SCALE_PER_CHANNEL ? a.v_scale + (size_t)h * D : nullptr;
#pragma unroll 1
      for (int c0 = grp * (D / 2); c0 < (grp + 1) * (D / 2); c0 += whole ? 32 : 16) {
        uint32_t w[4][4];
        if (whole) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float x[16];
            channels(c0 + 16 * hh, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 s = vs_ch ? *reinterpret_cast<const float2*>(vs_ch + c0 + 16 * hh + 2 * i) : make_float2(1.0f, 1.0f);
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * i] * s.x, x[2 * i + 1] * s.y);
              w[2 * hh + i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
        } else {
          float x[16];
          channels(c0, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __float_as_uint(x[i]);
        }
        dev::quad_transpose(w);
        // piece k is now this lane's 16 bytes of the quad's row k (out_dim is a
        // multiple of 8: whole pieces)
        const bool in = !whole || c0 + 8 * (lane & 3) < a.out_dim;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at[k] && in)
            *reinterpret_cast<uint4*>(at[k] + (whole ? 2 : 4) * c0 + 16 * (lane & 3)) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
      }
      ptx::tc_fence_before();
    }
  }

  // every role ends here; TMEM is released once no warp can touch it
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DT, int D, bool SPLIT, bool CAP, bool FOLD>
cudaError_t launch_tree_tile(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeArgs& a, int grid, size_t smem,
                             cudaStream_t stream) {
  static std::atomic<int> smem_set[64];
  const void* kernel = reinterpret_cast<const void*>(tree_tile_kernel<DT, D, SPLIT, CAP, FOLD>);
  if (cudaError_t e = raise_smem_limit(kernel, smem_set, smem)) return e;
  return launch_pdl(tree_tile_kernel<DT, D, SPLIT, CAP, FOLD>, grid, kTtWarps * 32, smem, stream, tk, tv, a);
}

template <int DT, int D, bool CAP>
cudaError_t dispatch_tree_tile(bool split, bool fold, const CUtensorMap& tk, const CUtensorMap& tv,
                               const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  if constexpr (D == 256) {
    if (split) return launch_tree_tile<DT, D, true, CAP, false>(tk, tv, a, grid, smem, stream);
  } else {
    if (split && fold) return launch_tree_tile<DT, D, true, CAP, true>(tk, tv, a, grid, smem, stream);
    if (split) return launch_tree_tile<DT, D, true, CAP, false>(tk, tv, a, grid, smem, stream);
  }
  if (fold) return launch_tree_tile<DT, D, false, CAP, true>(tk, tv, a, grid, smem, stream);
  return launch_tree_tile<DT, D, false, CAP, false>(tk, tv, a, grid, smem, stream);
}

template <int DT, int D>
cudaError_t dispatch_tree_tile(bool split, bool fold, const CUtensorMap& tk, const CUtensorMap& tv,
                               const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  return a.softcap > 0.0f ? dispatch_tree_tile<DT, D, true>(split, fold, tk, tv, a, grid, smem, stream)
                          : dispatch_tree_tile<DT, D, false>(split, fold, tk, tv, a, grid, smem, stream);
}

}  // namespace kvq
