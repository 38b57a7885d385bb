// key_mass_tc.cuh -- kvq_key_mass for many query rows per kv head (17..128 a
// launch: drafts x GQA group, or the last tokens of a prompt) on the tcgen05
// tensor cores.
//
// What key_mass.cuh computes, with 128 keys as the MMA's M dimension and the
// rows (padded to NR, a multiple of 32) as N:
//
//   S [128 keys x NR] = K [128 keys x D] . Q [NR x D]^T      A = K in TMEM, B = Q (f16, shared)
//   weight of a key   = sum over its row of S of exp2(S alpha_r - c_r)
//
// so a key's weight is a sum along one thread's TMEM columns: no exchange
// between lanes.  K and S are double-buffered in TMEM (2 x D/2 and 2 x 128
// columns: all of it at head_dim 256), Q stays in shared memory for the whole
// piece, and a K tile's codes never leave shared memory but into TMEM.  A
// per-channel K scale's second Q part (SPLIT, see key_mass.cuh) is a second
// pass of the MMAs into the same S.
//
// Warp roles (14 warps):
//   0-7   weights: warp w takes lane quarter w & 3 (32 keys, one a thread) and
//         half w >> 2 of the rows; also the Q prologue of each piece.  The two
//         halves of a key meet in shared memory, in a fixed order.
//   8-11  K dequant: one key row per thread -> f16 K columns in TMEM
//   12    TMA producer of the code stages (shared with decode.cuh)
//   13    TMEM allocation; issues the MMAs
#pragma once

#include "decode_tc.cuh"

namespace kvq {

// A query row's rule in shared memory, for tiles that some row does not see
// whole or that reach past some row's position.
struct __align__(16) MassTcRule {
  int begin, end, pos, d0;
};

// CAP: a softcap (in instances of its own: fourteen warps share the instruction
// caches, and everything that made the weight loop's code larger -- the cap
// beside it, prefetching or unrolling over more columns -- cost 10 to 25%).
template <int DT, int D, bool SPLIT, bool CAP>
__global__ void __launch_bounds__(kMassTcWarps * 32, 1)
    key_mass_tc_kernel(const __grid_constant__ CUtensorMap tmk, const DecodeArgs a, const MassArgs ms, const int NR) {
  using Gm = Geo<DT, D, kTcKeys>;
  constexpr int KT = kTcKeys;
  constexpr int kDqK = 8, kProducer = 12, kMma = 13;
  constexpr int K_COL = 0, S_COL = D;  // K: 2 x D/2 columns, S: 2 x 128
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* base = smem_raw + pad;
  const MassTcSmem lay = mass_tc_layout(D, NR, SPLIT, a.stages, a.batch, a.stage_stride);
  uint8_t* ring = base + lay.ring;
  uint8_t* q_s = base + lay.q;                                       // [parts][D/64 slabs][NR rows][128 B]
  const uint32_t q_part = (uint32_t)NR * D * 2;
  float2* r_ac = reinterpret_cast<float2*>(base + lay.rows);         // [NR] logit factor, log-sum-exp
  float2* r_ne = r_ac + NR;                                          // [NR] bias per key, pos - d0 - k0
  MassTcRule* r_rule = reinterpret_cast<MassTcRule*>(r_ne + NR);     // [NR]
  float* half_sum = reinterpret_cast<float*>(r_rule + NR);           // [2][KT] the second half's sums
  float* k_scale = half_sum + 2 * KT;                                // [4][KT] K scales of tile it, at it & 3
  int* pl_pre = reinterpret_cast<int*>(base + lay.pre);
  int* pl_misc = pl_pre + a.batch + 1;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(base + lay.bars);
  uint64_t* bar_empty = bar_full + a.stages;
  uint64_t* b_s = bar_empty + a.stages;  // [2] MMAs of tile it complete: S written, K columns it & 1 free
  uint64_t* b_sfree = b_s + 2;           // [2] S buffer read
  uint64_t* b_kfull = b_s + 4;           // [2] K tile in TMEM
  uint64_t* b_qfull = b_s + 6;           // Q of a piece written
  uint64_t* b_ksc = b_s + 7;             // [4] K scales of tile it in k_scale slot it & 3 (per-row K)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_s + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&bar_full[s], 1);
      ptx::mbar_init(&bar_empty[s], 4);  // K dequant warps
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&b_s[i], 1);
      ptx::mbar_init(&b_sfree[i], 8);
      ptx::mbar_init(&b_kfull[i], 4);
    }
    ptx::mbar_init(b_qfull, 8);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&b_ksc[i], 4);
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
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!ptx::mbar_try_wait(bar, parity)) dev::wait_or_abort(bar, parity, abort_flag, a.err);
  };
  const bool k_row = a.k_mode == KVQ_SCALE_PER_ROW;

  if (warp == kProducer) {
    // ============================================================ producer
    produce_lanes<Gm>(a, sp, &tmk, &tmk, ring, bar_full, bar_empty, pl_pre, pl_misc);
  } else if (warp >= kDqK && warp < kDqK + 4) {
    // ========================================================== K dequant
    const int q = warp - kDqK, kk = 32 * q + lane;
    const uint32_t t_k = tmem + ((uint32_t)(32 * q) << 16) + K_COL;
    constexpr int HCH = Gm::NCH / 2;             // 16-byte chunks of a channel half
    constexpr int CW = DT == KVQ_INT4 ? 16 : 8;  // K columns per chunk
    uint32_t it = 0;
    RingPos rp;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      for (int key0 = k0; key0 < k1; key0 += KT, ++it, rp.next(a.stages)) {
        wait(&bar_full[rp.stage], rp.phase);
        const uint8_t* st = ring + (size_t)rp.stage * a.stage_stride;
        const uint32_t buf = it & 1;
        // the key's whole code row (and scale) first, so that the stage goes
        // back to the producer at once
        uint4 w[2 * HCH];
#pragma unroll
        for (int jj = 0; jj < 2 * HCH; ++jj) {
          const uint32_t byte = (uint32_t)jj * 16;
          w[jj] = *reinterpret_cast<const uint4*>(
              st + (byte / Gm::SPAN) * (KT * Gm::SPAN) + dev::swz<Gm::SPAN>(kk * Gm::SPAN + byte % Gm::SPAN));
        }
        // the scale for the weight warps: slot it & 3 was last read for tile
        // it - 4, before the MMAs of tile it - 2 that this warp waits for below
        float ksv = 1.0f;
        if (k_row) ksv = reinterpret_cast<const float*>(st + Gm::CODE_BYTES)[kk];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bar_empty[rp.stage]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[HCH * CW];
#pragma unroll
          for (int jj = 0; jj < HCH; ++jj) dev::k_cols<DT>(w[half * HCH + jj], v + CW * jj);
          if (half == 0 && it >= 2) wait(&b_s[buf], ((it - 2) >> 1) & 1);  // the MMAs two tiles back are done
          ptx::tc_fence_after();
          if constexpr (HCH * CW == 64)
            ptx::tmem_st64(t_k + (D / 2) * buf + 64 * half, v);
          else
            ptx::tmem_st32(t_k + (D / 2) * buf + 32 * half, v);
        }
        if (k_row) k_scale[(it & 3) * KT + kk] = ksv;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&b_kfull[buf]);
          if (k_row) ptx::mbar_arrive(&b_ksc[it & 3]);
        }
      }
    }
  } else if (warp == kMma) {
    // ================================================================ MMA
    const uint32_t idesc = (1u << 4) | ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    const uint64_t q_desc = ptx::smem_desc_sw128(ptx::smem_u32(q_s));
    const uint32_t q_lo = (uint32_t)q_desc, d_hi = (uint32_t)(q_desc >> 32);
    const uint32_t slab = ((uint32_t)NR * 128) >> 4, part = q_part >> 4;
    uint32_t it = 0;
    int pc = 0;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next, ++pc) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      for (int key0 = k0; key0 < k1; key0 += KT, ++it) {
        const uint32_t buf = it & 1;
        if (key0 == k0) wait(b_qfull, pc & 1);
        wait(&b_kfull[buf], (it >> 1) & 1);
        if (it >= 2) wait(&b_sfree[buf], ((it - 2) >> 1) & 1);
        __syncwarp();
        ptx::tc_fence_after();
        const uint32_t s_col = tmem + S_COL + 128 * buf, k_col = tmem + K_COL + (D / 2) * buf;
#pragma unroll 1
        for (int p = SPLIT ? 1 : 0; p >= 0; --p) {  // the small part first: less is rounded
#pragma unroll 1
          for (int sl = 0; sl < D / 64; ++sl)
            ptx::mma_f16_ts_x4(s_col, k_col + 32 * sl, 8, q_lo + p * part + sl * slab, d_hi, idesc,
                               sl > 0 || (SPLIT && p == 0) ? 1u : 0u);
        }
        ptx::mma_commit(&b_s[buf]);
      }
    }
    if (it > 0) {
      // every MMA has completed before TMEM can be released
      const uint32_t last = it - 1;
      if (!ptx::mbar_wait_bounded(&b_s[last & 1], (last >> 1) & 1) && lane == 0) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ============================================================ weights
    const int q = warp & 3, side = warp >> 2, kk = 32 * q + lane;
    const uint32_t t_s = tmem + ((uint32_t)(32 * q) << 16) + S_COL;
    const int G = a.group, Hq = a.num_q_heads;
    const float inv_g = __frcp_rn((float)G);
    const float softcap = a.softcap, inv_cap = softcap > 0.0f ? 1.0f / softcap : 1.0f;
    const float cap_l2 = softcap * kLog2e;
    constexpr int LPR = D / 8, RPP = 32 / LPR;  // lanes per row (8 channels each), rows per warp pass
    const int rsub = lane / LPR, cl = lane % LPR;
    uint32_t it = 0;
    for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next) {
      int b, h, k0, k1, L, u;
      sp.piece(a, gt, b, h, k0, k1, L, u, next);
      const VSeq vs = a.vseq[b];
      const int rows = vs.ntok * G;
      // every warp has read the previous piece's rows (and waited for its last
      // MMAs, so the Q operand is free)
      ptx::named_bar_sync(5, 256);
      // ---- the piece's row rules (a thread a row; its loads run while the
      // operand below is made) and Q operand
      float2 ac = make_float2(0.0f, INFINITY), ne = make_float2(0.0f, 0.0f);
      MassTcRule ru{0, 0, 0, 0};
      bool live = false;
      if (tid < rows) {
        const int t = dev::div_small(tid, inv_g), hq = h * G + tid - t * G;
        const size_t tok = (size_t)vs.tok0 + t;
        const float lse = ms.lse[tok * Hq + hq];
        const dev::RowRule rr = dev::row_rule(a, tok, vs.pos0 + t, hq, L);
        live = rr.begin < rr.end && lse != -INFINITY;
        if (live) {
          // lse less the anchor's bias: in fp64, both may be large
          const double s = a.slopes ? (double)a.slopes[hq] * (double)rr.d0 : 0.0;
          ac.y = (float)(((double)lse + s) * 1.4426950408889634);
          ne = make_float2(rr.ns, (float)(rr.pos - rr.d0 - k0));
          ru = MassTcRule{rr.begin, rr.end, rr.pos, rr.d0};
        }
      }
      {
        const bool kc = a.k_mode == KVQ_SCALE_PER_CHANNEL;
        float ksv[8];
        int ek = 0;
        if (kc) {
          const float4* ksp = reinterpret_cast<const float4*>(a.k_scale + (size_t)h * D + 8 * cl);
          const float4 s0 = __ldg(ksp), s1 = __ldg(ksp + 1);
          ksv[0] = s0.x; ksv[1] = s0.y; ksv[2] = s0.z; ksv[3] = s0.w;
          ksv[4] = s1.x; ksv[5] = s1.y; ksv[6] = s1.z; ksv[7] = s1.w;
          float km = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) km = fmaxf(km, fabsf(ksv[i]));
          km = ptx::redux_max(km);
          ek = km > 0.0f ? min(126, max(-126, dev::ceil_log2(km))) : 0;
          const float sk = dev::pow2i(-ek);
#pragma unroll
          for (int i = 0; i < 8; ++i) ksv[i] *= sk;
        }
        float fac = a.sm_scale;
        if (a.k_mode == KVQ_SCALE_PER_TENSOR) fac *= a.k_scale[0];
        fac *= softcap > 0.0f ? inv_cap : kLog2e;
        constexpr int BAT = 4;  // row loads in flight
#pragma unroll 1
        for (int r0 = warp * RPP + rsub; r0 < NR; r0 += BAT * 8 * RPP) {
          uint4 raw[BAT];
#pragma unroll
          for (int i = 0; i < BAT; ++i) {
            const int r = r0 + i * 8 * RPP, t = dev::div_small(r, inv_g);
            raw[i] = r < rows ? ptx::ldg_nc_v4(a.q + (((size_t)vs.tok0 + t) * Hq + h * G + r - t * G) * D + 8 * cl)
                              : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < BAT; ++i) {
            const int r = r0 + i * 8 * RPP;
            float qv[8];
            const uint32_t ww[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              qv[2 * j] = __uint_as_float(ww[j] << 16);
              qv[2 * j + 1] = __uint_as_float(ww[j] & 0xFFFF0000u);
            }
            if (kc) {
#pragma unroll
              for (int j = 0; j < 8; ++j) qv[j] *= ksv[j];
            }
            float qm = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) qm = ptx::max_nan(qm, fabsf(qv[j]));
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) qm = ptx::max_nan(qm, __shfl_xor_sync(0xffffffffu, qm, o));
            const int eq = qm > 0.0f ? min(126, max(-126, dev::ceil_log2(qm))) : 0;
            const float sq = dev::pow2i(-eq);
            uint32_t w[4], lo[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float x0, x1;
              if constexpr (DT == KVQ_INT4) {
                const float f = (m & 1) ? sq * dev::odd_channel_factor<DT>() : sq;  // channels m, m + 4
                x0 = qv[m] * f;
                x1 = qv[m + 4] * f;
              } else {
                x0 = qv[2 * m] * sq;
                x1 = qv[2 * m + 1] * sq;
              }
              w[m] = dev::pack_h2(x0, x1);
              lo[m] = dev::rest_h2(x0, x1, w[m]);
            }
            if (r < NR) {
              uint8_t* dst = q_s + (cl >> 3) * (NR * 128) + r * 128 + ((((uint32_t)cl & 7u) ^ ((uint32_t)r & 7u)) << 4);
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
              if constexpr (SPLIT) *reinterpret_cast<uint4*>(dst + q_part) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              if (cl == 0) {
                const int e = ek + eq, e1 = e / 2;
                const float al = fminf(fac * dev::pow2i(e1) * dev::pow2i(e - e1), 3.4028234e38f);
                // (a row with an infinity or a NaN is marked: see below)
                r_ac[r].x = qm <= 3.4028234e38f ? al : __uint_as_float(0x7FC00000u);
              }
            }
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(b_qfull);
      }
      ptx::named_bar_sync(5, 256);  // the logit factors are visible
      if (tid < NR) {
        // a row that is padding, sees nothing or has no weight: factor 0 and
        // log-sum-exp +inf give it a weight of exactly 0 everywhere.  Times 0
        // its scores may still be NaN, when its query holds an infinity or a
        // NaN: an interval that ends at 0 then keeps every tile of the piece
        // on the slow path, which selects by the rules.
        if (!live) {
          const float al = r_ac[tid].x;
          if (al != al) ru.begin = -1;
          r_ac[tid].x = 0.0f;
        }
        r_ac[tid].y = ac.y;
        r_ne[tid] = ne;
        r_rule[tid] = ru;
      }
      ptx::named_bar_sync(5, 256);  // the rows are visible
      // tiles inside [bmax, emin) and, under a bias, at or below pmin need no
      // mask and have linear distances for every row
      int bmax = 0, emin = 0x7FFFFFFF, pmin = 0x7FFFFFFF;
      for (int r = lane; r < rows; r += 32) {
        const MassTcRule ru = r_rule[r];
        if (ru.begin < ru.end) {
          bmax = max(bmax, ru.begin);
          emin = min(emin, ru.end);
          pmin = min(pmin, ru.pos);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        bmax = max(bmax, __shfl_xor_sync(0xffffffffu, bmax, o));
        emin = min(emin, __shfl_xor_sync(0xffffffffu, emin, o));
        pmin = min(pmin, __shfl_xor_sync(0xffffffffu, pmin, o));
      }
      const bool bias = a.slopes != nullptr;
      const int32_t* bt = a.block_table + (size_t)vs.brow * a.max_blocks_per_seq;
      const int c_lo = side * (NR / 2), c_hi = c_lo + NR / 2;

      // the page of this thread's next key is looked up a tile ahead
      int id_next = side == 0 && k0 + kk < k1 ? bt[(k0 + kk) >> a.log2_bs] : -1;
      for (int key0 = k0; key0 < k1; key0 += KT, ++it) {
        const uint32_t buf = it & 1;
        const int key = key0 + kk;
        float* out = nullptr;
        float old = 0.0f;
        const int id = id_next;
        if (side == 0 && key + KT < k1) id_next = bt[(key + KT) >> a.log2_bs];
        if (side == 0 && key < k1) {
          if (id >= 0 && id < a.num_blocks) {
            out = ms.mass + ((size_t)id * a.num_kv_heads + h) * a.block_size + (key & (a.block_size - 1));
            // (scaled where it is used: the load stays in flight until then)
            if (ms.decay != 0.0f && key < vs.len - ms.fresh) old = *out;
          }
        }
        float ks = 1.0f;
        if (k_row) {
          wait(&b_ksc[it & 3], (it >> 2) & 1);
          ks = k_scale[(it & 3) * KT + kk];
        }
        wait(&b_s[buf], (it >> 1) & 1);
        ptx::tc_fence_after();
        const bool fast = key0 >= bmax && key0 + KT <= emin && (!bias || key0 + KT - 1 <= pmin);
        const float kf = (float)(key - k0);
        // (K scale times logit factor first: a product of codes and a large scale
        // may leave fp32's range where the logit does not)
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_hi; c0 += 16) {
          float y[16];
          dev::tmem_ld_cols<16>(t_s + 128 * buf + c0, y);
          if (fast) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 ac = *reinterpret_cast<const float4*>(r_ac + c0 + i);
              float x0, x1;
              if constexpr (CAP) {
                x0 = fmaf(cap_l2, dev::tanh_near(y[i] * (ks * ac.x)), -ac.y);
                x1 = fmaf(cap_l2, dev::tanh_near(y[i + 1] * (ks * ac.z)), -ac.w);
              } else {
                x0 = fmaf(y[i], ks * ac.x, -ac.y);
                x1 = fmaf(y[i + 1], ks * ac.z, -ac.w);
              }
              if (bias) {
                const float4 ne = *reinterpret_cast<const float4*>(r_ne + c0 + i);
                x0 = fmaf(ne.x, ne.y - kf, x0);
                x1 = fmaf(ne.z, ne.w - kf, x1);
              }
              s0 += ptx::fast_exp2(x0);
              s1 += ptx::fast_exp2(x1);
            }
          } else {
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
              const float2 ac = r_ac[c0 + i], ne = r_ne[c0 + i];
              const MassTcRule ru = r_rule[c0 + i];
              float x = y[i] * (ks * ac.x);
              if constexpr (CAP) x = cap_l2 * dev::tanh_near(x);
              if (bias) x = fmaf(ne.x, (float)(abs(ru.pos - key) - ru.d0), x);
              s0 += key >= ru.begin && key < ru.end ? ptx::fast_exp2(x - ac.y) : 0.0f;
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b_sfree[buf]);
        // one barrier a tile between a key's two warps: the second half's sums
        // are written again two tiles on, behind the next tile's barrier
        s0 += s1;
        if (side == 1) half_sum[buf * KT + kk] = s0;
        ptx::named_bar_sync(1 + q, 64);
        if (out) *out = ms.decay * old + (s0 + half_sum[buf * KT + kk]);
      }
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

template <int DT, int D, bool SPLIT, bool CAP>
cudaError_t launch_key_mass_tc_d(const CUtensorMap& tk, const DecodeArgs& a, const MassArgs& m, int nr, int grid,
                                 size_t smem, cudaStream_t stream) {
  static std::atomic<int> smem_set[64];
  const void* kernel = reinterpret_cast<const void*>(key_mass_tc_kernel<DT, D, SPLIT, CAP>);
  if (cudaError_t e = raise_smem_limit(kernel, smem_set, smem)) return e;
  return launch_pdl(key_mass_tc_kernel<DT, D, SPLIT, CAP>, grid, kMassTcWarps * 32, smem, stream, tk, a, m, nr);
}

// head_dim 128 or 256, any K scale mode but PER_GROUP.
template <int DT>
cudaError_t dispatch_key_mass_tc(int head_dim, const CUtensorMap& tk, const DecodeArgs& a, const MassArgs& m, int nr,
                                 int grid, size_t smem, cudaStream_t stream) {
  const bool split = a.k_mode == KVQ_SCALE_PER_CHANNEL, cap = a.softcap > 0.0f;
  auto go = [&](auto dtag, auto stag) -> cudaError_t {
    constexpr int d = decltype(dtag)::value;
    constexpr bool s = decltype(stag)::value;
    return cap ? launch_key_mass_tc_d<DT, d, s, true>(tk, a, m, nr, grid, smem, stream)
               : launch_key_mass_tc_d<DT, d, s, false>(tk, a, m, nr, grid, smem, stream);
  };
  auto by_split = [&](auto dtag) -> cudaError_t {
    return split ? go(dtag, std::true_type{}) : go(dtag, std::false_type{});
  };
  if (head_dim == 256) return by_split(std::integral_constant<int, 256>{});
  if (head_dim == 128) return by_split(std::integral_constant<int, 128>{});
  return cudaErrorInvalidValue;
}

}  // namespace kvq
