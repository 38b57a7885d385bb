// tree_tile.cuh -- attention of many drafted nodes per kv head over the
// quantized paged cache on the tcgen05 tensor cores: kvq_attend_tree from 17
// query rows on at head_dim 128 and 256.
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
// and the output.  P overwrites its own S, so that head_dim 256 has two S
// buffers too (Q 128 + O 256 + S 2 x 64 columns) and QK^T of the next tile runs
// during the softmax; one warp issues both products, whose order in the tensor
// pipe is what keeps S, P and Q apart.
//
// Warp roles (16 warps): 0-3 softmax, one thread a row (Q of a piece into
// TMEM, S -> P with lazy row maxima, the epilogue); 4-7 K dequant, key
// 32 (w & 1) + lane, channel half w >> 1; 8-11 V dequant, the same; 12 TMA
// producer of the code stages; 13 the MMAs.
#pragma once

#include "decode_tc.cuh"

namespace kvq {

namespace dev {

// Address of 16-byte f16 chunk c of key row kk in an f16 tile: 64-element slabs
// of [kTile rows][128 B] in the tensor core's 128-byte swizzle.
template <int SLAB>
__device__ __forceinline__ uint32_t tt_chunk(uint32_t tile, int kk, int c) {
  return tile + (uint32_t)(c >> 3) * SLAB + (uint32_t)kk * 128u + ((((uint32_t)c & 7u) ^ ((uint32_t)kk & 7u)) << 4);
}

// One 16-byte chunk of a V code row in k_cols's order; e4m3 by the hardware
// conversion with NaN codes (a key no row sees may hold one) made finite.
template <int DT>
__device__ __forceinline__ void tt_v_cols(const uint4 w4, uint32_t* v) {
  if constexpr (DT == KVQ_FP8_E4M3) {
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = f8cvt(w[i], 0x4410u);
      v[2 * i + 1] = f8cvt(w[i], 0x4432u);
    }
  } else {
    k_cols<DT>(w4, v);
  }
}

// Transposes the 4 x 4 16-byte pieces of a quad of lanes: x[k] of lane i
// becomes what x[i] of lane k was (i, k within the quad).
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4][4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? x[k][i] : x[k + 1][i], 1);
      (odd ? x[k][i] : x[k + 1][i]) = got;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? x[k][i] : x[k + 2][i], 2);
      (high ? x[k][i] : x[k + 2][i]) = got;
    }
  }
}

}  // namespace dev

// SPLIT: the Q operand in two f16 parts (a per-channel K scale and an lse that
// is asked for).  At head_dim 128 the second part has tensor-memory columns of
// its own and a second pass of QK^T adds into the same S; at head_dim 256 a
// unit then has at most 64 rows, the second parts are the operand's rows
// 64..127, and warps 2 and 3 hand their rows of S to warps 0 and 1 through
// shared memory (as f16: 2^-11 of a 2^-12 correction).  CAP: a softcap.
template <int DT, int D, bool SPLIT, bool CAP>
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
  constexpr int kDqK = 4, kDqV = 8, kProducer = 12, kMma = 13;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  const TtSmem lay = tt_smem_layout(D, a.stages, a.batch, a.stage_stride, STACK);
  uint8_t* ring = base + lay.ring;
  const uint32_t kf = ptx::smem_u32(base + lay.kf), vf = ptx::smem_u32(base + lay.vf);
  float* ksb = reinterpret_cast<float*>(base + lay.sc);  // [4][KT] K scales of tile it, at it & 3
  float* vsb = ksb + 4 * KT;                              // [4][KT] its V scales over 2^F
  int* fexp = reinterpret_cast<int*>(vsb + 4 * KT);       // [4] its F
  int* pl_pre = reinterpret_cast<int*>(base + lay.pre);
  int* pl_misc = pl_pre + a.batch + 1;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(base + lay.bars);
  uint64_t* bar_empty = bar_full + a.stages;
  uint64_t* b_s = bar_empty + a.stages;  // [2] QK^T of tile it complete: S buffer and K tile it & 1
  uint64_t* b_kfull = b_s + 2;           // [2] K f16 tile written
  uint64_t* b_vfull = b_s + 4;           // [2] V f16 tile written
  uint64_t* b_p = b_s + 6;               // [2] P of tile it written (and O rescaled)
  uint64_t* b_pv = b_s + 8;              // [2] PV of tile it complete: V tile it & 1 free
  uint64_t* b_q = b_s + 10;              // Q of a piece in TMEM
  uint64_t* b_ksc = b_s + 11;            // [4] K scales of tile it (per-row K)
  uint64_t* b_vsc = b_s + 15;            // [4] V scales of tile it (per-row V)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + lay.slot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&bar_full[s], 1);
      ptx::mbar_init(&bar_empty[s], 8);  // K and V dequant warps
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&b_s[i], 1);
      ptx::mbar_init(&b_kfull[i], 4);
      ptx::mbar_init(&b_vfull[i], 4);
      ptx::mbar_init(&b_p[i], 4);
      ptx::mbar_init(&b_pv[i], 1);
    }
    ptx::mbar_init(b_q, 4);
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&b_ksc[i], 2);  // the two warps of channel half 0
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

  if (warp == kProducer) {
    // ============================================================ producer
    ptx::regs_down<96>();
    produce_lanes<Gm, true, true>(a, sp, &tmk, &tmv, ring, bar_full, bar_empty, pl_pre, pl_misc);
  } else if (warp >= kDqK && warp < kDqV + 4) {
    // ==================================================== K and V dequant
    // A stage's codes are converted 64 bytes of a row at a time; the wait for
    // the MMA that frees the f16 tile comes before the first store.
    ptx::regs_down<104>();
    const bool is_v = warp >= kDqV;
    const int q = warp - (is_v ? kDqV : kDqK);
    const int kk = 32 * (q & 1) + lane, hf = q >> 1;
    constexpr int HB = Gm::DP / 2;                       // code bytes of a channel half
    constexpr int PB = HB < 64 ? HB : 64;                // of a piece
    constexpr int NC = PB / 16;                          // its 16-byte chunks
    constexpr int CW = DT == KVQ_INT4 ? 16 : 8;          // f16 pairs per chunk
    const uint32_t f16_base = is_v ? vf : kf;
    uint64_t* b_free = is_v ? b_pv : b_s;
    uint64_t* b_full = is_v ? b_vfull : b_kfull;
    const uint32_t code_off = is_v ? (uint32_t)Gm::CODE_BYTES : 0u;
    const bool scaled = is_v ? v_row : k_row;
    uint32_t it = 0;
    RingPos rp;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      int F = -126;  // V-scale normaliser exponent of the piece
      const int first_key = a.vseq[b].lo;  // (a row below it may hold anything)
      for (int key0 = Order::first(k0, k1); Order::more(key0, k0, k1); key0 += Order::step, ++it, rp.next(a.stages)) {
        const uint32_t buf = it & 1;
        wait(&bar_full[rp.stage], rp.phase);
        const uint8_t* st = ring + (size_t)rp.stage * a.stage_stride;
        if (scaled && hf == 0) {
          // K: slot it & 3 was last read by the softmax of tile it - 4, done
          // before PV of that tile was issued, which was before QK^T of it - 2;
          // this warp waited for QK^T of it - 3 and waits here for it - 2.
          // V: the softmax of it - 4 was done before PV of it - 3 completed,
          // which this warp waited for on its previous tile.
          const float* scp = reinterpret_cast<const float*>(st + 2 * Gm::CODE_BYTES + (is_v ? KT * 4 : 0));
          float sc = scp[kk];
          if (is_v) {
            auto seen = [&](int key) { return key >= first_key && key < L; };
            float vm = seen(key0 + lane) ? scp[lane] : 0.0f;
            if (seen(key0 + 32 + lane)) vm = fmaxf(vm, scp[32 + lane]);
            vm = ptx::redux_max(vm);
            if (vm > 0.0f) F = max(F, min(126, max(-126, dev::ceil_log2(vm))));
            vsb[(it & 3) * KT + kk] = seen(key0 + kk) ? sc * dev::pow2i(-F) : 0.0f;
            if (q == 0 && lane == 0) fexp[it & 3] = F;
          } else {
            if (it >= 2) wait(&b_free[buf], ((it - 2) >> 1) & 1);
            ksb[(it & 3) * KT + kk] = sc;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(is_v ? &b_vsc[it & 3] : &b_ksc[it & 3]);
        }
        const uint32_t tile = f16_base + buf * TILE;
#pragma unroll
        for (int pc = 0; pc < HB / PB; ++pc) {
          uint4 w[NC];
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const uint32_t byte = (uint32_t)(hf * HB + pc * PB + 16 * j);
            w[j] = *reinterpret_cast<const uint4*>(st + code_off + (byte / Gm::SPAN) * (KT * Gm::SPAN) +
                                                   dev::swz<Gm::SPAN>((uint32_t)kk * Gm::SPAN + byte % Gm::SPAN));
          }
          if (pc == HB / PB - 1) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bar_empty[rp.stage]);
          }
          uint32_t v[NC * CW];
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            if (is_v) dev::tt_v_cols<DT>(w[j], v + CW * j);
            else dev::k_cols<DT>(w[j], v + CW * j);
          }
          if (pc == 0 && it >= 2) wait(&b_free[buf], ((it - 2) >> 1) & 1);  // the MMA two tiles back has read this tile
#pragma unroll
          for (int c = 0; c < NC * CW / 4; ++c) {
            const uint32_t addr = dev::tt_chunk<SLAB>(tile, kk, hf * (D / 16) + pc * (NC * CW / 4) + c);
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
    // QK^T(it + 1), PV(it), QK^T(it + 2), ...: executed in this order, so the
    // S buffer of it + 2 is written after PV(it) has read its P there.
    ptx::regs_down<96>();
    constexpr uint32_t idesc_qk = ptx::idesc_f16_f32(128, KT);
    constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, D) | (1u << 16);  // B MN-major
    const uint64_t kd = ptx::smem_desc_sw128(kf);
    const uint32_t k_lo = (uint32_t)kd, d_hi = (uint32_t)(kd >> 32);
    const uint32_t v_lo = (uint32_t)ptx::smem_desc_sw128_mn(vf, SLAB);
    auto issue_qk = [&](uint32_t j) {
      const uint32_t buf = j & 1;
      wait(&b_kfull[buf], (j >> 1) & 1);
      __syncwarp();
      ptx::tc_fence_after();
      if constexpr (SPLIT && !STACK) {
        // the small part first: less is rounded
#pragma unroll
        for (int sl = 0; sl < D / 64; ++sl)
          ptx::mma_f16_ts_x4(tmem + S_COL + KT * buf, tmem + QL_COL + 32 * sl, 8, k_lo + ((buf * TILE + sl * SLAB) >> 4),
                             d_hi, idesc_qk, sl > 0 ? 1u : 0u);
      }
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl)
        ptx::mma_f16_ts_x4(tmem + S_COL + KT * buf, tmem + Q_COL + 32 * sl, 8, k_lo + ((buf * TILE + sl * SLAB) >> 4),
                           d_hi, idesc_qk, sl > 0 || (SPLIT && !STACK) ? 1u : 0u);
      ptx::mma_commit(&b_s[buf]);
    };
    // a piece's first PV overwrites O
    auto issue_pv = [&](uint32_t j, bool first) {
      const uint32_t buf = j & 1;
      wait(&b_vfull[buf], (j >> 1) & 1);
      wait(&b_p[buf], (j >> 1) & 1);
      __syncwarp();
      ptx::tc_fence_after();
      ptx::mma_f16_ts_x4_step(tmem + O_COL, tmem + S_COL + KT * buf, 8, v_lo + buf * (TILE >> 4), (16 * 128) >> 4, d_hi,
                              idesc_pv, first ? 0u : 1u);
      ptx::mma_commit(&b_pv[buf]);
    };
    uint32_t it = 0;
    int pc = 0;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next, ++pc) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      wait(b_q, pc & 1);
      issue_qk(it);
      for (int key0 = Order::first(k0, k1); Order::more(key0, k0, k1); key0 += Order::step, ++it) {
        if (Order::more(key0 + Order::step, k0, k1)) issue_qk(it + 1);
        issue_pv(it, key0 == Order::first(k0, k1));
      }
    }
    // every MMA has completed before TMEM can be released
    if (it > 0 && !ptx::mbar_wait_bounded_inl(&b_pv[(it - 1) & 1], ((it - 1) >> 1) & 1) && lane == 0)
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    __syncwarp();
  } else if (warp < kDqK) {
    // ============================================================ softmax
    ptx::regs_up<208>();
    const int q = warp;
    // query row = TMEM lane (STACK: lanes 64..127 hold the second parts of rows 0..63)
    const int r = STACK ? (32 * q + lane) & 63 : 32 * q + lane;
    const bool second = STACK && q >= 2;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16);
    const int G = a.group, Hq = a.num_q_heads, rows = a.rows;
    const uint32_t exch = ptx::smem_u32(base + lay.exch);
    // S of the second parts, [2][64 rows][KT keys] f16, 16-byte chunks XOR (row & 7)
    auto exch_at = [&](uint32_t buf, int chunk) -> uint32_t {
      return exch + buf * (64 * KT * 2) + (uint32_t)r * (KT * 2) + (((uint32_t)chunk ^ ((uint32_t)r & 7u)) << 4);
    };
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
      float alpha = 1.0f;
      // ---- Q of this piece (every QK^T of the previous one has completed: this
      // thread waited for its last S): the per-channel K scale folded in under a
      // power-of-two normaliser, the row normalised by the power of two at or
      // above its maximum, f16 pairs in the K order of the K tile.
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
        constexpr int NCH8 = D / 8, BAT = 16;
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
        for (int c32 = 0; c32 < D / 32; ++c32) {
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
        // (a row with no node sees the piece's keys: finite scores that feed
        // only its own unwritten output)
        ru.end = L;
        ru.bits = -1;
        if (valid) ru = dev::row_rule<true>(a, tok, vs.pos0 + t_row, hq, L);
        ptx::tc_fence_before();
        __syncwarp();
      }
      if (lane == 0) ptx::mbar_arrive(b_q);

      // tanh(x) = x P(x^2) for |x| <= kCapNear, P the minimax polynomial of
      // degree 3 to tanh(sqrt t) / sqrt t there (1.5e-7 relative); x = alpha S
      constexpr float kCapNear = 0.35f;
      const float cap2 = CAP ? a.softcap * kLog2e : 0.0f, al2 = alpha * alpha;
      const float c0f = alpha * cap2, c1f = -0.33332422f * al2 * c0f, c2f = 0.13295799f * al2 * al2 * c0f,
                  c3f = -0.04895823f * al2 * al2 * al2 * c0f;
      const float cap_near =
          CAP && alpha > 6e-5f && alpha < 1.6e4f && cap2 > 1e-6f && cap2 < 1e6f ? kCapNear / alpha : -1.0f;
      const ptx::f32x2 aa = ptx::pack_x2(alpha, alpha);

      float mu = -INFINITY;         // reference maximum of this row (log2 units)
      ptx::f32x2 l2 = ptx::pack_x2(0.0f, 0.0f);  // its weight sum, in two halves (even and odd keys)
      int F = -126;                 // V-scale normaliser exponent
      for (int key0 = Order::first(k0, k1); Order::more(key0, k0, k1); key0 += Order::step, ++it) {
        const bool first = key0 == Order::first(k0, k1);
        const uint32_t buf = it & 1;
        const uint32_t s_col = t_lane + S_COL + KT * buf;
        wait(&b_s[buf], (it >> 1) & 1);
        if (idle) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&b_p[buf]);
          continue;
        }
        ptx::tc_fence_after();
        if constexpr (STACK) {
          // one barrier a tile between a row's two warps (q & 1 and 2 + (q & 1)):
          // a buffer is written again two tiles on, after the other side has
          // passed the barrier of the tile between
          if (second) {
            float y[KT];
            dev::tmem_ld_cols<KT>(s_col, y);
#pragma unroll
            for (int c8 = 0; c8 < KT / 8; ++c8)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(exch_at(buf, c8)),
                           "r"(dev::pack_h2(y[8 * c8], y[8 * c8 + 1])), "r"(dev::pack_h2(y[8 * c8 + 2], y[8 * c8 + 3])),
                           "r"(dev::pack_h2(y[8 * c8 + 4], y[8 * c8 + 5])), "r"(dev::pack_h2(y[8 * c8 + 6], y[8 * c8 + 7]))
                           : "memory");
            ptx::named_bar_sync(1 + (q & 1), 64);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&b_p[buf]);
            continue;
          }
          ptx::named_bar_sync(1 + (q & 1), 64);
        }
        if (k_row) wait(&b_ksc[it & 3], (it >> 2) & 1);
        const float* ksc = ksb + (it & 3) * KT;
        const float* vsc = vsb + (it & 3) * KT;
        const bool full = key0 >= ru.begin && key0 + KT <= ru.end;
        uint32_t bits[2] = {0u, 0u};  // visible keys of a tile that is not whole
        if (!full) {
          dev::tree_sees_64(a, ru, key0, bits);
          const int lo = min(KT, max(0, ru.begin - key0)), hi = min(KT, max(0, ru.end - key0));
          if (lo < hi) {
            const uint64_t in = (hi == 64 ? ~0ull : (1ull << hi) - 1) & ~((1ull << lo) - 1);
            bits[0] |= (uint32_t)in;
            bits[1] |= (uint32_t)(in >> 32);
          }
        }
        // Scores (with a per-row K scale in): 64 keys in registers; under a cap,
        // whose unrolled code would not stay in the instruction cache, 32 at a
        // time, twice.
        constexpr int CH = CAP ? 32 : KT;
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
          if constexpr (STACK) {
#pragma unroll
            for (int c8 = 0; c8 < CH / 8; ++c8) {
              uint32_t w[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                           : "r"(exch_at(buf, c0 / 8 + c8))
                           : "memory");
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                y[8 * c8 + 2 * j] += f.x;
                y[8 * c8 + 2 * j + 1] += f.y;
              }
            }
          }
          if (k_row) {
#pragma unroll
            for (int k = 0; k < CH; k += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(ksc + c0 + k);
              ptx::mul_x2(y[k], y[k + 1], y[k], y[k + 1], s4.x, s4.y);
              ptx::mul_x2(y[k + 2], y[k + 3], y[k + 2], y[k + 3], s4.z, s4.w);
            }
          }
        };
        auto hide = [&](int c0) {
#pragma unroll
          for (int k = 0; k < CH; ++k)
            if (!((bits[CAP ? c0 / 32 : k / 32] >> (k % 32)) & 1u)) y[k] = -INFINITY;
        };
        float m = -INFINITY, least = INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < KT; c0 += CH) {
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
        const bool near = CAP && fmaxf(fabsf(m), fabsf(least)) <= cap_near;
        if constexpr (CAP) {
          if (near) {
            const float t = m * m;
            m *= fmaf(fmaf(fmaf(c3f, t, c2f), t, c1f), t, c0f);
          } else if (m != -INFINITY) {
            float x[2] = {m * alpha, 0.0f};
            dev::cap_scores<2>(x, cap2);
            m = x[0];
          }
        } else {
          m *= alpha;
        }
        float fs = 1.0f;  // growth of the V-scale normaliser
        if (v_row) {
          wait(&b_vsc[it & 3], (it >> 2) & 1);
          const int fn = fexp[it & 3];
          if (fn > F) {
            fs = (F - fn < -126) ? 0.0f : dev::pow2i(F - fn);
            F = fn;
          }
        }
        // move the reference only when the tile's maximum exceeds it by more
        // than 8 (P <= 2^8 in f16); a row with no key yet holds zeros in O
        float corr = 1.0f;
        bool resc = false;
        if (m > mu + 8.0f) {
          if (mu != -INFINITY) {
            corr = ptx::fast_exp2(mu - m);
            resc = !first;
          }
          mu = m;
        }
        l2 = ptx::mul_x2(l2, ptx::pack_x2(corr, corr));
        resc = resc || (fs != 1.0f && !first);
        if (__any_sync(0xffffffffu, resc)) {
          // bring this warp's rows of O to the new reference and normaliser
          // (after the previous PV has landed)
          wait(&b_pv[(it - 1) & 1], ((it - 1) >> 1) & 1);
          ptx::tc_fence_after();
          const float f = resc ? corr * fs : 1.0f;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            dev::tmem_ld_cols<16>(t_lane + O_COL + c0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            dev::tmem_st_cols<16>(t_lane + O_COL + c0, o);
          }
        }
        // P = 2^(y - mu), with the V scales, f16 pairs; the sums take the fp32
        // weights
        const float nmu = mu == -INFINITY ? 0.0f : -mu;
        const ptx::f32x2 nm = ptx::pack_x2(nmu, nmu);
        auto weigh = [&](int c0, auto&& score) {
          uint32_t p[CH / 2];
#pragma unroll
          for (int k = 0; k < CH; k += 2) {
            float z0, z1;
            ptx::unpack_x2(score(ptx::pack_x2(y[k], y[k + 1])), z0, z1);
            const ptx::f32x2 e = ptx::pack_x2(ptx::fast_exp2(z0), ptx::fast_exp2(z1));
            l2 = ptx::add_x2(l2, e);
            float e0, e1;
            ptx::unpack_x2(e, e0, e1);
            if (v_row) {
              const float2 s2 = *reinterpret_cast<const float2*>(vsc + c0 + k);
              ptx::mul_x2(e0, e1, e0, e1, s2.x, s2.y);
            }
            p[k / 2] = dev::pack_h2(e0, e1);
          }
          // (the columns of S that P takes have been read: P is half as wide)
          __syncwarp();
          if constexpr (CH == 32) ptx::tmem_st16(s_col + c0 / 2, *reinterpret_cast<uint32_t(*)[16]>(p));
          else ptx::tmem_st32(s_col, p);
        };
        if constexpr (!CAP) {
          weigh(0, [&](ptx::f32x2 x) { return ptx::fma_x2(x, aa, nm); });
        } else {
          const ptx::f32x2 cc0 = ptx::pack_x2(c0f, c0f), cc1 = ptx::pack_x2(c1f, c1f), cc2 = ptx::pack_x2(c2f, c2f),
                           cc3 = ptx::pack_x2(c3f, c3f);
#pragma unroll 1
          for (int c0 = 0; c0 < KT; c0 += CH) {
            load_s(c0);
            if (!near) {
#pragma unroll
              for (int k = 0; k < CH; k += 2) ptx::mul_x2(y[k], y[k + 1], y[k], y[k + 1], alpha, alpha);
              dev::cap_scores<CH>(y, cap2);
              if (!full) hide(c0);
            }
            // near: y P(y^2) - mu, the factors of alpha in P's coefficients (a
            // row with hidden keys, of score -inf, is not near); else y - mu
            const bool nr = near;
            weigh(c0, [&](ptx::f32x2 x) {
              if (!nr) return ptx::add_x2(x, nm);
              const ptx::f32x2 t = ptx::mul_x2(x, x);
              return ptx::fma_x2(x, ptx::fma_x2(ptx::fma_x2(ptx::fma_x2(t, cc3, cc2), t, cc1), t, cc0), nm);
            });
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b_p[buf]);
      }

      // ---- epilogue: O out of TMEM, normalised.  The workspace and the output
      // are written after the preceding grid (the producer waited for it before
      // the first tile's codes).  A unit of one piece (`whole`) is finished here:
      // head sink, static V scale and bf16, as in the combine; otherwise the
      // partial with its base-2 log-sum-exp.
      if (it > 1) wait(&b_pv[it & 1], ((it - 2) >> 1) & 1);
      wait(&b_pv[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (idle || second) continue;
      ptx::tc_fence_after();
      float l, lb;
      ptx::unpack_x2(l2, l, lb);
      l += lb;
      float inv = l > 0.0f ? (v_row ? dev::pow2i(F) : 1.0f) / l : 0.0f;
      const bool whole = k0 == (vs.lo & ~(KT - 1)) && k1 == L;
      // channels c0 .. c0 + 15 of this thread's row, in channel order
      auto channels = [&](int c0, float (&x)[16]) {
        float o[16];
        dev::tmem_ld_cols<16>(t_lane + O_COL + c0, o);
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
        if (l > 0.0f) {
          lse = (mu + ptx::fast_log2(l)) * 0.69314718055994530942f;
          if (a.head_sink && valid) inv /= 1.0f + expf(a.head_sink[hq] - lse);
        }
        if (a.v_mode == KVQ_SCALE_PER_TENSOR) inv *= a.v_scale[0];
        if (valid && a.lse_out) a.lse_out[tok * Hq + hq] = lse;
        dst = reinterpret_cast<unsigned long long>(a.out + (tok * Hq + hq) * a.out_dim);
      } else {
        if (valid) a.part_lse[(size_t)u * rows + r] = l > 0.0f ? mu + ptx::fast_log2(l) : -INFINITY;
        dst = reinterpret_cast<unsigned long long>(a.part_o + ((size_t)u * rows + r) * D);
      }
      // quads of lanes store 64 bytes of a row at a time
      if (!valid) dst = 0;
      unsigned long long at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, dst, (lane & ~3) | i);
      const float* vs_ch = whole && a.v_mode == KVQ_SCALE_PER_CHANNEL ? a.v_scale + (size_t)h * D : nullptr;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += whole ? 32 : 16) {
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
  } else {
    ptx::regs_down<96>();
  }

  // every role ends here; TMEM is released once no warp can touch it
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DT, int D, bool SPLIT, bool CAP>
cudaError_t launch_tree_tile(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeArgs& a, int grid, size_t smem,
                             cudaStream_t stream) {
  static std::atomic<int> smem_set[64];
  const void* kernel = reinterpret_cast<const void*>(tree_tile_kernel<DT, D, SPLIT, CAP>);
  if (cudaError_t e = raise_smem_limit(kernel, smem_set, smem)) return e;
  return launch_pdl(tree_tile_kernel<DT, D, SPLIT, CAP>, grid, kTtWarps * 32, smem, stream, tk, tv, a);
}

template <int DT>
cudaError_t dispatch_tree_tile(int head_dim, bool split, const CUtensorMap& tk, const CUtensorMap& tv,
                               const DecodeArgs& a, int grid, size_t smem, cudaStream_t stream) {
  const bool cap = a.softcap > 0.0f;
  if (head_dim == 128) {
    if (split) return cap ? launch_tree_tile<DT, 128, true, true>(tk, tv, a, grid, smem, stream) : launch_tree_tile<DT, 128, true, false>(tk, tv, a, grid, smem, stream);
    return cap ? launch_tree_tile<DT, 128, false, true>(tk, tv, a, grid, smem, stream) : launch_tree_tile<DT, 128, false, false>(tk, tv, a, grid, smem, stream);
  }
  if (head_dim == 256) {
    if (split) return cap ? launch_tree_tile<DT, 256, true, true>(tk, tv, a, grid, smem, stream) : launch_tree_tile<DT, 256, true, false>(tk, tv, a, grid, smem, stream);
    return cap ? launch_tree_tile<DT, 256, false, true>(tk, tv, a, grid, smem, stream) : launch_tree_tile<DT, 256, false, false>(tk, tv, a, grid, smem, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
