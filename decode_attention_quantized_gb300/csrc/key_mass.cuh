// key_mass.cuh -- the attention weight that every cached key receives, added up
// (kvq_key_mass): for each key j and kv head, sum over the call's query rows of
// exp(s_j - lse_row), onto what the key held before.
//
// The scores are the attention's own (same operands, scales, cap, bias and
// mask), the row's log-sum-exp is given, so one pass over the K codes is all:
// no running maximum, no V, no partials.  Same split plan, producer and
// 64-key stages as decode.cuh with the K side only (the LATENT layout of a
// stage); four consumer warps of 16 keys each, keys as MMA-M and query rows as
// MMA-N, so a key's sum over rows is a sum over a thread's accumulators and two
// shuffles, and each key is written by one lane: no atomics, one fixed order.
//
// The result is fp32 and has to agree with fp32 scores: codes are exact in
// f16 and so are bf16 queries, but a query with a per-channel K scale folded in
// is not; there the operand is split into two f16 values (two MMAs).  The cap
// takes a tanh of small relative error, the masked attention's (50 * tanh(x / 50)
// from 1 - 2 / (e^2x + 1) would be 2e-5 off).
#pragma once

#include "decode.cuh"
#include "score_rule.cuh"

namespace kvq {

// SPLIT: a per-channel K scale (two-part Q operand).  GRP: per-group K scales.
template <int DT, int D, int NT, bool SPLIT, bool GRP>
__global__ void __launch_bounds__(kMassThreads, NT == 1 && D <= 256 ? (SPLIT ? 3 : 4) : (NT <= 4 ? 2 : 1))
    key_mass_kernel(const __grid_constant__ CUtensorMap tmk, const DecodeArgs a, const MassArgs ms) {
  using Gm = Geo<DT, D>;
  constexpr float kLog2e = 1.4426950408889634f;
  // the Q operand(s) in shared memory: all but one n-tile of at most 256
  // channels, whose fragments stay in registers
  constexpr bool QS = NT > 1 || D > 256;
  constexpr int ROWS = 8 * NT;
  constexpr int CH = DT == KVQ_INT4 ? 32 : 16;  // channels of a 16-byte code chunk
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;
  uint8_t* q_smem = ring + (size_t)a.stages * a.stage_stride;
  constexpr size_t kQBytes = QS ? (size_t)ROWS * D * 2 : 0;
  MassRow* rows_s = reinterpret_cast<MassRow*>(q_smem + kQBytes * (SPLIT ? 2 : 1));
  int* pl_pre = reinterpret_cast<int*>(rows_s + ROWS);
  int* pl_misc = pl_pre + a.batch + 1;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(pl_misc + 4 + ((a.batch + 5) & 1));
  uint64_t* bar_empty = bar_full + a.stages;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&bar_full[s], 1);
      ptx::mbar_init(&bar_empty[s], kMassWarps);
    }
    ptx::fence_mbar_init();
  }
  const Slice<kTile, true> sp = build_slice<kTile, true>(a, pl_pre, pl_misc);
  if (warp == kMassWarps) {
    produce_lanes<Gm>(a, sp, &tmk, &tmk, ring, bar_full, bar_empty, pl_pre, pl_misc);
    return;
  }

  const uint32_t q_base = ptx::smem_u32(q_smem);
  // byte offset of Q[row][k]: 2D-byte rows, the low three bits of the 16-byte
  // chunk index XOR (row & 7)
  auto q_off = [](int row, int k) -> uint32_t {
    return (uint32_t)(row * 2 * D + ((((k >> 3) & ~7) | (((k >> 3) ^ row) & 7)) << 4) + (k & 7) * 2);
  };
  const int g = lane >> 2, c = lane & 3, G = a.group;
  const float inv_g = __frcp_rn((float)G);
  const int ld_key = ((lane >> 3) & 1) * 8 + (lane & 7);
  const int ld_chunk = lane >> 4;
  const bool k_row = a.k_mode == KVQ_SCALE_PER_ROW;
  const float softcap = a.softcap;
  const float cap_l2 = softcap * kLog2e;
  const int ng = a.sk_n;
  const int gmask = GRP ? (1 << a.log2_gs) - 1 : 0;
  RingPos rp;
  bool ok = true;

  for (int gt = sp.t_begin, next; gt < sp.t_end; gt = next) {
    int b, h, k0, k1, L, slot;
    sp.piece(a, gt, b, h, k0, k1, L, slot, next);
    const VSeq vs = a.vseq[b];
    const int rows = vs.ntok * G;

    // ---- the piece's query rows: operand and rule
    uint32_t qf[QS ? 1 : Gm::NMT][2], ql[SPLIT && !QS ? Gm::NMT : 1][2];
    ptx::named_bar_sync(1, kMassWarps * 32);  // the previous piece's rows are read
    // (a thread a row; its loads run while the operand is made)
    MassRow mr{};
    if (tid < rows) {
      const int t = dev::div_small(tid, inv_g), hq = h * G + tid - t * G;
      const size_t tok = (size_t)vs.tok0 + t;
      const float lse = ms.lse[tok * a.num_q_heads + hq];
      const dev::RowRule ru = dev::row_rule(a, tok, vs.pos0 + t, hq, L);
      // lse less the anchor's bias: in fp64, both may be large
      const double s = a.slopes ? (double)a.slopes[hq] * (double)ru.d0 : 0.0;
      mr.c = (float)(((double)lse + s) * 1.4426950408889634);
      mr.ns = ru.ns;
      mr.begin = ru.begin;
      mr.end = lse == -INFINITY ? 0 : ru.end;  // a row without weight
      mr.pos = ru.pos;
      mr.d0 = ru.d0;
    }
#pragma unroll 1
    for (int nt = QS ? warp : 0; nt < NT; nt += QS ? kMassWarps : 1) {
      const int row = nt * 8 + g;
      uint32_t f[Gm::NMT][2], lo[SPLIT ? Gm::NMT : 1][2];
      float al = dev::q_prologue<DT, D, SPLIT>(a, row, (size_t)vs.tok0, rows, h, c, f, lo);
      if constexpr (QS) {
#pragma unroll
        for (int ks = 0; ks < Gm::NMT; ++ks) {
          ptx::st_shared_u32(q_base + q_off(row, ks * 16 + 2 * c), f[ks][0]);
          ptx::st_shared_u32(q_base + q_off(row, ks * 16 + 8 + 2 * c), f[ks][1]);
          if constexpr (SPLIT) {
            ptx::st_shared_u32(q_base + (uint32_t)kQBytes + q_off(row, ks * 16 + 2 * c), lo[ks][0]);
            ptx::st_shared_u32(q_base + (uint32_t)kQBytes + q_off(row, ks * 16 + 8 + 2 * c), lo[ks][1]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < Gm::NMT; ++ks) {
          qf[ks][0] = f[ks][0];
          qf[ks][1] = f[ks][1];
          if constexpr (SPLIT) {
            ql[ks][0] = lo[ks][0];
            ql[ks][1] = lo[ks][1];
          }
        }
      }
      if (c == 0 && (QS || warp == 0)) {
        if (softcap > 0.0f) al = fminf(al / softcap, 3.4028234e38f);
        rows_s[row].alpha = al;
      }
    }
    ptx::named_bar_sync(1, kMassWarps * 32);
    if (tid < ROWS) {
      mr.alpha = tid < rows ? rows_s[tid].alpha : 0.0f;
      rows_s[tid] = mr;
    }
    ptx::named_bar_sync(1, kMassWarps * 32);

    const int32_t* bt = a.block_table + (size_t)vs.brow * a.max_blocks_per_seq;
    // the page of this warp's next sub-tile is looked up a tile ahead
    int id_next = k0 + warp * kSub < k1 ? bt[(k0 + warp * kSub) >> a.log2_bs] : -1;
    for (int key0 = k0; key0 < k1; key0 += kTile, rp.next(a.stages)) {
      const int kb = key0 + warp * kSub;
      const int key_a = kb + g, key_b = key_a + 8;
      const int id = id_next;
      if (kb + kTile < k1) id_next = bt[(kb + kTile) >> a.log2_bs];
      // where this sub-tile's weights live (its 16 keys share a page), and
      // what they held
      float* out = nullptr;
      float old_a = 0.0f, old_b = 0.0f;
      if (kb < k1) {
        if (id >= 0 && id < a.num_blocks)
          out = ms.mass + ((size_t)id * a.num_kv_heads + h) * a.block_size + (kb & (a.block_size - 1));
        if (out && c == 0 && ms.decay != 0.0f) {
          if (key_a < k1 && key_a < vs.len - ms.fresh) old_a = out[g];
          if (key_b < k1 && key_b < vs.len - ms.fresh) old_b = out[g + 8];
        }
      }
      if (ok) {
        ok = ptx::mbar_wait_bounded_inl(&bar_full[rp.stage], rp.phase);
        if (!ok) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
      }
      const uint8_t* st = ring + (size_t)rp.stage * a.stage_stride;
      const uint32_t sk_base = ptx::smem_u32(st);
      const float* ks_row = reinterpret_cast<const float*>(st + Gm::CODE_BYTES);
      float sum_a = 0.0f, sum_b = 0.0f;
      if (ok && out) {
        // ---- S = K Q^T: 16 keys x 8 NT rows, each code converted once
        float acc[NT][4], gx[GRP ? NT : 1][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
#pragma unroll
        for (int nt = 0; nt < (GRP ? NT : 1); ++nt) gx[nt][0] = gx[nt][1] = gx[nt][2] = gx[nt][3] = 0.0f;
        // one n-tile: odd k-steps accumulate apart, so that the MMAs do not
        // wait on one another
        float odd[NT == 1 ? 4 : 1] = {};
        const uint32_t row_off = (uint32_t)(warp * kSub + ld_key) * Gm::SPAN;
        auto step = [&](const uint32_t (&A)[4], int ks) {
          if constexpr (!QS) {
            if (ks & 1) ptx::mma_16816(odd, A, qf[ks][0], qf[ks][1]);
            else ptx::mma_16816(acc[0], A, qf[ks][0], qf[ks][1]);
            if constexpr (SPLIT) {
              if (ks & 1) ptx::mma_16816(acc[0], A, ql[ks][0], ql[ks][1]);
              else ptx::mma_16816(odd, A, ql[ks][0], ql[ks][1]);
            }
          } else {
            const int mi = lane >> 3;
#pragma unroll
            for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
              const uint32_t qb = q_base + (uint32_t)(part * kQBytes);
#pragma unroll
              for (int np = 0; np < NT / 2; ++np) {
                uint32_t R[4];
                ptx::ldmatrix_x4(R, qb + q_off((2 * np + (mi >> 1)) * 8 + (lane & 7), ks * 16 + (mi & 1) * 8));
                ptx::mma_16816(acc[2 * np], A, R[0], R[1]);
                ptx::mma_16816(acc[2 * np + 1], A, R[2], R[3]);
              }
              if constexpr (NT == 1) {
                uint32_t R[2];
                ptx::ldmatrix_x2(R, qb + q_off(lane & 7, ks * 16 + (mi & 1) * 8));
                if (ks & 1) ptx::mma_16816(odd, A, R[0], R[1]);
                else ptx::mma_16816(acc[0], A, R[0], R[1]);
              }
            }
          }
        };
#pragma unroll
        for (int kk = 0; kk < Gm::NCH / 2; ++kk) {
          const uint32_t byte = (uint32_t)(2 * kk + ld_chunk) * 16;
          uint32_t R[4];
          ptx::ldmatrix_x4(R, sk_base + (byte / Gm::SPAN) * (kTile * Gm::SPAN) +
                                  dev::swz<Gm::SPAN>(row_off + byte % Gm::SPAN));
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const int j = 2 * kk + h2;
#pragma unroll
            for (int t = 0; t < (DT == KVQ_INT4 ? 2 : 1); ++t) {
              uint32_t A[4];
              dev::k_frag<DT>(R[2 * h2], R[2 * h2 + 1], t, A);
              step(A, DT == KVQ_INT4 ? 2 * j + t : j);
            }
            if (GRP && (((j + 1) * CH) & gmask) == 0) {
              const int grp = (((j + 1) * CH) >> a.log2_gs) - 1;
              const float ga = ks_row[(warp * kSub + g) * ng + grp], gb = ks_row[(warp * kSub + g + 8) * ng + grp];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float v = acc[nt][e];
                  if constexpr (NT == 1) {
                    v += odd[e];
                    odd[e] = 0.0f;
                  }
                  gx[GRP ? nt : 0][e] = fmaf(v, e < 2 ? ga : gb, gx[GRP ? nt : 0][e]);
                  acc[nt][e] = 0.0f;
                }
            }
          }
        }
        float ksa = 1.0f, ksb = 1.0f;
        if (k_row) {
          ksa = ks_row[warp * kSub + g];
          ksb = ks_row[warp * kSub + g + 8];
        }
        // ---- weights: element e -> key a (e < 2) or b, row 2c + (e & 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const MassRow r = rows_s[nt * 8 + 2 * c + i];
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int e = 2 * e2 + i, key = e2 ? key_b : key_a;
              float s = GRP ? gx[GRP ? nt : 0][e] : acc[nt][e];
              if constexpr (NT == 1 && !GRP) s += odd[e];
              float x = s * r.alpha * (e2 ? ksb : ksa);
              if (softcap > 0.0f) x = cap_l2 * dev::tanh_near(x);
              if (a.slopes) x = fmaf(r.ns, (float)(abs(r.pos - key) - r.d0), x);
              const float p = key >= r.begin && key < r.end ? ptx::fast_exp2(x - r.c) : 0.0f;
              if (e2) sum_b += p; else sum_a += p;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bar_empty[rp.stage]);
      sum_a += __shfl_xor_sync(0xffffffffu, sum_a, 1);
      sum_b += __shfl_xor_sync(0xffffffffu, sum_b, 1);
      sum_a += __shfl_xor_sync(0xffffffffu, sum_a, 2);
      sum_b += __shfl_xor_sync(0xffffffffu, sum_b, 2);
      if (out && ok && c == 0) {
        if (key_a < k1) out[g] = ms.decay * old_a + sum_a;
        if (key_b < k1) out[g + 8] = ms.decay * old_b + sum_b;
      }
    }
  }
}

template <int DT, int D, int NT, bool SPLIT, bool GRP>
cudaError_t key_mass_d(const CUtensorMap* tk, const DecodeArgs* a, const MassArgs* m, int grid, size_t smem,
                       cudaStream_t stream, int* blocks_per_sm) {
  static std::atomic<int> smem_set[64];
  const void* kernel = reinterpret_cast<const void*>(key_mass_kernel<DT, D, NT, SPLIT, GRP>);
  if (cudaError_t e = raise_smem_limit(kernel, smem_set, smem)) return e;
  if (blocks_per_sm)
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, key_mass_kernel<DT, D, NT, SPLIT, GRP>,
                                                         kMassThreads, smem);
  return launch_pdl(key_mass_kernel<DT, D, NT, SPLIT, GRP>, grid, kMassThreads, smem, stream, *tk, *a, *m);
}

template <int DT>
cudaError_t dispatch_key_mass(int head_dim, int nt, int k_mode, const CUtensorMap* tk, const DecodeArgs* a,
                              const MassArgs* m, int grid, size_t smem, cudaStream_t stream, int* blocks_per_sm) {
  auto by_nt = [&](auto dtag, auto split, auto grp) -> cudaError_t {
    constexpr int d = decltype(dtag)::value;
    constexpr bool s = decltype(split)::value, g = decltype(grp)::value;
    switch (nt) {
      case 1: return key_mass_d<DT, d, 1, s, g>(tk, a, m, grid, smem, stream, blocks_per_sm);
      case 2: return key_mass_d<DT, d, 2, s, g>(tk, a, m, grid, smem, stream, blocks_per_sm);
      case 4: return key_mass_d<DT, d, 4, s, g>(tk, a, m, grid, smem, stream, blocks_per_sm);
      case 8:
        if constexpr (d <= 256) return key_mass_d<DT, d, 8, s, g>(tk, a, m, grid, smem, stream, blocks_per_sm);
        return cudaErrorInvalidValue;
      default: return cudaErrorInvalidValue;
    }
  };
  auto by_mode = [&](auto dtag) -> cudaError_t {
    if (k_mode == KVQ_SCALE_PER_CHANNEL) return by_nt(dtag, std::true_type{}, std::false_type{});
    if constexpr (decltype(dtag)::value <= 256)
      if (k_mode == KVQ_SCALE_PER_GROUP) return by_nt(dtag, std::false_type{}, std::true_type{});
    return by_nt(dtag, std::false_type{}, std::false_type{});
  };
  switch (head_dim) {
    case 64: return by_mode(std::integral_constant<int, 64>{});
    case 128: return by_mode(std::integral_constant<int, 128>{});
    case 256: return by_mode(std::integral_constant<int, 256>{});
    case 576:
      if constexpr (DT != KVQ_INT4) return by_mode(std::integral_constant<int, 576>{});
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
