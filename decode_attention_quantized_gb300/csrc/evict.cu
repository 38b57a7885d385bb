// evict.cu -- eviction from the paged cache by accumulated attention weight:
// which rows of a (sequence, kv head) stay (kvq_evict_select), and the moving
// of those rows to the front of the sequence's pages (kvq_evict_compact).
#include "kvq_internal.h"
#include "ptx.cuh"

namespace kvq {
namespace {

// ------------------------------------------------------------------ select
//
// The `need` largest of M weights with ties to the lower index, in ascending
// index order: a radix select of the threshold (the weight as an ordered
// 32-bit key, four digits of 8 bits from the top, a histogram of the keys that
// still match), then one ordered pass that writes every row above the
// threshold and the first rows equal to it.
//
// A cluster of CTAs holds one (sequence, kv head): each warp reads a
// contiguous stretch of the weights from global memory once and keeps it in
// registers, so the passes touch no memory but the histogram.  Weights of one
// head share a few exponents and may all be equal, so a histogram has a column
// per lane (bank = lane): no two lanes of a warp ever meet, whatever the
// values (with one 2048-bin histogram a CTA and its collisions the select of
// 4 x 262,144 rows took 118 us, that of 512 heads of up to 131,072 rows
// 1356 us).  The columns' sums meet through the cluster's shared memory, where
// every CTA adds them up for itself: one cluster barrier a digit.  Integer
// adds: their order cannot show.

constexpr int kSelWarps = kSelThreads / 32;

// Ascending keys of ascending weights: -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256 * 32];     // [bin][lane]
  __shared__ uint32_t total[2][256];      // this CTA's counts of a digit (two passes' worth)
  __shared__ uint32_t s_gt[kSelWarps], s_eq[kSelWarps], s_scan[8], s_digit[2], s_cta[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cs = ptx::cluster_size(), rank = ptx::cluster_rank();
  const int seg = (int)(blockIdx.x / cs);
  const int b = seg / a.num_kv_heads, h = seg - b * a.num_kv_heads;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const int raw = a.seq_lens[b];
  const int L = raw < 0 ? 0 : (raw > a.lim ? a.lim : raw);
  if (raw != L && h == 0 && rank == 0 && tid == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
  int32_t* keep = a.keep + (size_t)seg * a.budget;
  const int n = min(L, a.budget);
  if (h == 0 && rank == 0 && tid == 0) a.kept_lens[b] = n;
  // everything stays, or only the protected ends do (the whole cluster agrees)
  const int need_all = a.budget - a.sinks - a.recent;
  const bool whole = L <= a.budget;
  if (whole || need_all == 0) {
    for (int i = (int)rank * kSelThreads + tid; i < a.budget; i += (int)cs * kSelThreads)
      keep[i] = i >= n ? -1 : (whole || i < a.sinks ? i : L - a.budget + i);
    return;
  }
  for (int i = (int)rank * kSelThreads + tid; i < a.sinks + a.recent; i += (int)cs * kSelThreads) {
    if (i < a.sinks) keep[i] = i;
    else keep[need_all + i] = L - a.recent + (i - a.sinks);
  }

  // this warp's stretch of the M rows between the ends: [w0, w0 + m), the
  // stretches in (CTA, warp) order
  const int M = L - a.sinks - a.recent;
  const int warps = (int)cs * kSelWarps;
  const int stretch = ((M + warps - 1) / warps + 31) & ~31;
  const long long w0l = (long long)((int)rank * kSelWarps + warp) * stretch;
  const int w0 = (int)(w0l < M ? w0l : M);
  const int m = min(M, w0 + stretch) - w0;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks_per_seq;
  bool bad = false;
  auto load = [&](int i) -> uint32_t {  // row w0 + i; branch-free, so that loads run ahead
    const int pos = a.sinks + w0 + i;
    const int id = bt[pos >> a.log2_bs];
    const bool fine = (unsigned)id < (unsigned)a.num_blocks;
    bad = bad || !fine;
    const float* p = a.mass + (fine ? ((size_t)id * a.num_kv_heads + h) * a.block_size + (pos & (a.block_size - 1)) : 0);
    const uint32_t k = order_key(*p);
    return fine ? k : 0u;
  };
  // the first kSelKeys x 32 rows of the stretch in registers, a longer
  // stretch's rest read again in each pass
  uint32_t key[kSelKeys];
#pragma unroll
  for (int j = 0; j < kSelKeys; ++j) key[j] = 0u;
#pragma unroll
  for (int j0 = 0; j0 < kSelKeys; j0 += 8) {
    if (j0 * 32 < m) {
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) {
        const int i = min(j * 32 + lane, m - 1);
        key[j] = load(i);
      }
    }
  }
  // f(index in the stretch, key) for each of this lane's rows
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
      if (j * 32 < m) {
        if (j * 32 + lane < m) f(key[j]);
      }
    }
    for (int i = kSelKeys * 32 + lane; i < m; i += 32) f(load(i));
  };

  uint32_t prefix = 0;
  int need = need_all;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256 * 32 / 4; i += kSelThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (pass == 0)
      each([&](uint32_t k) { atomicAdd(&hist[(k >> 24) * 32 + lane], 1u); });
    else
      each([&](uint32_t k) {
        if ((k >> shift) >> 8 == prefix) atomicAdd(&hist[((k >> shift) & 255u) * 32 + lane], 1u);
      });
    __syncthreads();
    {
      // two threads a bin, sixteen columns each, starting apart by bin so that
      // a warp's lanes read different banks
      const int bin = tid >> 1, c0 = (tid & 1) * 16;
      uint32_t s = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += hist[bin * 32 + c0 + ((j + bin) & 15)];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      if ((tid & 1) == 0) total[pass & 1][bin] = s;
    }
    ptx::cluster_sync();
    // the cluster's counts, highest bin first, and the scan that finds the digit
    if (tid < 256) {
      const int bin = 255 - tid;
      const uint32_t at = ptx::smem_u32(&total[pass & 1][bin]);
      uint32_t cnt = 0;
      for (uint32_t r = 0; r < cs; r += 4) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = r + j < cs ? ptx::ld_cluster_u32(at, r + j) : 0u;
        cnt += (v[0] + v[1]) + (v[2] + v[3]);
      }
      uint32_t incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_scan[warp] = incl;
      ptx::named_bar_sync(1, 256);
      uint32_t before = incl - cnt;  // keys in higher bins
      for (int w = 0; w < warp; ++w) before += s_scan[w];
      if (before < (uint32_t)need && before + cnt >= (uint32_t)need) {
        s_digit[0] = (uint32_t)bin;
        s_digit[1] = before;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | s_digit[0];
    need -= (int)s_digit[1];
  }
  if (bad) atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);

  // ---- ordered output
  const uint32_t T = prefix;  // `need` rows equal to it stay, the lowest
  uint32_t gt = 0, eq = 0;
  each([&](uint32_t k) {
    gt += k > T;
    eq += k == T;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t g = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      g += s_gt[w];
      e += s_eq[w];
    }
    s_cta[0] = g;
    s_cta[1] = e;
  }
  ptx::cluster_sync();
  uint32_t bg = 0, be = 0;  // rows above / equal before this warp's stretch
  if (lane < (int)rank) {
    bg = ptx::ld_cluster_u32(ptx::smem_u32(&s_cta[0]), (uint32_t)lane);
    be = ptx::ld_cluster_u32(ptx::smem_u32(&s_cta[1]), (uint32_t)lane);
  }
  if (lane < warp) {
    bg += s_gt[lane];
    be += s_eq[lane];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    bg += __shfl_xor_sync(0xffffffffu, bg, o);
    be += __shfl_xor_sync(0xffffffffu, be, o);
  }
  const uint32_t below = (1u << lane) - 1u;
  auto put = [&](int i0, uint32_t k) {  // rows i0 + lane of the stretch, whole warp
    const bool in = i0 + lane < m;
    const bool is_gt = in && k > T, is_eq = in && k == T;
    const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t g = bg + __popc(mg & below), e = be + __popc(me & below);
    if (is_gt || (is_eq && e < (uint32_t)need)) keep[a.sinks + g + min(e, (uint32_t)need)] = a.sinks + w0 + i0 + lane;
    bg += __popc(mg);
    be += __popc(me);
  };
#pragma unroll
  for (int j = 0; j < kSelKeys; ++j)
    if (j * 32 < m) put(j * 32, key[j]);
  for (int i0 = kSelKeys * 32; i0 < m; i0 += 32) put(i0, load(min(i0 + lane, m - 1)));
  ptx::cluster_sync();  // no CTA leaves while another reads its counts
}

// ----------------------------------------------------------------- compact
//
// Row i of a (sequence, kv head) becomes row keep[i] >= i (ascending): a
// gather of rows of Dp bytes and a dense, page-wise store, so bound by HBM
// (kept rows read once, written once).  The units are `rows` consecutive
// destination rows of one (sequence, kv head); a CTA takes units grid apart,
// one a round, through a ring of shared-memory stages: one bulk copy per row
// and side in (cp.async.bulk, completion on the stage's mbarrier; 4-byte
// scales and weights by cp.async beside them), one bulk copy per page run and
// side out.  Data never passes through registers, and the loads of the next
// rounds are in flight while a round waits and stores.
//
// In place, a unit's destination rows may hold rows that its own or an earlier
// unit of the same (sequence, kv head) has yet to read -- never a later one's,
// whose sources lie at or behind its own destination.  Units are numbered so
// that earlier chunks come in the same or an earlier round; a round's stores
// therefore wait until every CTA has loaded its unit of that round (a counter
// per round, all CTAs resident: a cooperative launch).  Every wait is bounded.

__global__ void __launch_bounds__(kCompactThreads) evict_compact_kernel(const CompactArgs a) {
  extern __shared__ __align__(128) uint8_t cmp_smem[];
  const int tid = threadIdx.x;
  __shared__ __align__(8) uint64_t bar[kCompactStages];
  __shared__ int s_ok;
  const int S = a.stages;
  if (tid == 0) {
    // every thread arrives twice: with its bulk bytes, and for its small copies
    for (int s = 0; s < S; ++s) ptx::mbar_init(&bar[s], 2 * kCompactThreads);
    ptx::fence_mbar_init();
    s_ok = 1;
  }
  __syncthreads();
  ptx::griddep_wait();
  const int segs = a.batch * a.num_kv_heads;
  const int rounds = (a.units + (int)gridDim.x - 1) / (int)gridDim.x;
  const int code_bytes = a.rows * a.row_bytes;  // one side of a stage
  const int nf = a.n_scale[0] + a.n_scale[1] + (a.mass ? 1 : 0);
  const int cap = a.max_blocks_per_seq << a.log2_bs;

  // unit of round k: its (sequence, kv head), first destination row and count
  // (0: nothing to move)
  auto unit = [&](int k, int& b, int& h, int& i0, int& n) {
    const long long u = (long long)k * gridDim.x + blockIdx.x;
    n = 0;
    b = h = i0 = 0;
    if (u >= a.units) return;
    const int chunk = (int)(u / segs), seg = (int)(u - (long long)chunk * segs);
    b = seg / a.num_kv_heads;
    h = seg - b * a.num_kv_heads;
    i0 = chunk << a.log2_rows;
    n = min(a.rows, min(a.kept_lens[b], a.budget) - i0);
    if (n <= 0) {
      n = 0;
      return;
    }
    // ascending rows whose last is in its place all are
    if (a.in_place && a.keep[(size_t)seg * a.budget + i0 + n - 1] == i0 + n - 1) n = 0;
  };
  // [block, kv head, row] index of position p of sequence b, or -1
  auto row_of = [&](const int32_t* table, int b, int h, int p, unsigned int flag) -> long long {
    if (p < 0 || p >= cap) {
      atomicOr(a.err, flag);
      return -1;
    }
    const int id = table[(size_t)b * a.max_blocks_per_seq + (p >> a.log2_bs)];
    if (id < 0 || id >= a.num_blocks) {
      atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
      return -1;
    }
    return ((long long)id * a.num_kv_heads + h) * a.block_size + (p & (a.block_size - 1));
  };

  auto issue = [&](int k) {
    const int s = k % S;
    uint8_t* st = cmp_smem + (size_t)s * a.stage_bytes;
    int b, h, i0, n;
    unit(k, b, h, i0, n);
    const int32_t* keep = a.keep + ((size_t)b * a.num_kv_heads + h) * a.budget + i0;
    // at most kCompactRows rows of two sides: kItems (row, side) pairs a thread
    constexpr int kItems = 2 * kCompactRows / kCompactThreads;
    long long src[kItems];
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int it = tid + i * kCompactThreads, r = it & (a.rows - 1);
      src[i] = -1;
      if (it < a.rows * a.sides && r < n) src[i] = row_of(a.block_table, b, h, keep[r], KVQ_DEVERR_KEEP_INDEX);
      if (src[i] >= 0) bytes += (uint32_t)a.row_bytes;
    }
    ptx::mbar_expect_tx(&bar[s], bytes);
    float* f = reinterpret_cast<float*>(st + a.sides * code_bytes);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (src[i] < 0) continue;
      const int it = tid + i * kCompactThreads, r = it & (a.rows - 1), side = it >> a.log2_rows;
      ptx::bulk_load(st + side * code_bytes + r * a.row_bytes, a.codes[side] + (size_t)src[i] * a.row_bytes,
                     (uint32_t)a.row_bytes, &bar[s]);
      const int ns = a.n_scale[side];
      for (int j = 0; j < ns; ++j)
        ptx::cp_async4(f + (side * a.n_scale[0] + j) * a.rows + r, a.scale[side] + (size_t)src[i] * ns + j);
      if (side == 0 && a.mass) ptx::cp_async4(f + (nf - 1) * a.rows + r, a.mass + src[i]);
    }
    ptx::cp_async_arrive(&bar[s]);
    ptx::mbar_arrive(&bar[s]);
  };

  for (int k = 0; k < S - 1 && k < rounds; ++k) issue(k);
  bool ok = true;
  for (int k = 0; k < rounds; ++k) {
    const int s = k % S;
    if (!ptx::mbar_wait_bounded(&bar[s], (uint32_t)(k / S) & 1u)) {
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
      s_ok = 0;
    }
    __syncthreads();  // the whole unit is in shared memory
    int b, h, i0, n;
    unit(k, b, h, i0, n);
    if (a.in_place) {
      if (tid == 0) {
        ptx::red_release_add(&a.round_count[k], 1u);
        if (n > 0 && s_ok) {
          const uint64_t t0 = ptx::globaltimer_ns();
          uint32_t i = 0;
          while (ptx::ld_acquire(&a.round_count[k]) < gridDim.x) {
            if ((++i & 63u) == 0u && ptx::globaltimer_ns() - t0 > ptx::kWaitLimitNs) {
              atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
              s_ok = 0;
              break;
            }
          }
        }
      }
      __syncthreads();
    }
    ok = s_ok != 0;
    if (n > 0 && ok) {
      const uint8_t* st = cmp_smem + (size_t)s * a.stage_bytes;
      // runs of rows in one destination page
      const int run = min(a.rows, a.block_size), runs = (n + run - 1) / run;
      asm volatile("fence.proxy.async;" ::: "memory");
      for (int it = tid; it < runs * a.sides; it += kCompactThreads) {
        const int side = it / runs, r0 = (it - side * runs) * run;
        const long long row = row_of(a.dst_table, b, h, i0 + r0, KVQ_DEVERR_KEEP_INDEX);
        if (row >= 0)
          ptx::bulk_store(a.codes[side] + (size_t)row * a.row_bytes, st + side * code_bytes + r0 * a.row_bytes,
                          (uint32_t)(min(run, n - r0) * a.row_bytes));
      }
      if (nf > 0) {
        const float* f = reinterpret_cast<const float*>(st + a.sides * code_bytes);
        for (int r = tid; r < n; r += kCompactThreads) {
          const long long row = row_of(a.dst_table, b, h, i0 + r, KVQ_DEVERR_KEEP_INDEX);
          if (row < 0) continue;
          for (int side = 0; side < a.sides; ++side)
            for (int j = 0; j < a.n_scale[side]; ++j)
              a.scale[side][(size_t)row * a.n_scale[side] + j] = f[(side * a.n_scale[0] + j) * a.rows + r];
          if (a.mass) a.mass[row] = f[(nf - 1) * a.rows + r];
        }
      }
    }
    ptx::bulk_commit();
    if (k + S - 1 < rounds) {
      // stage (k - 1) % S takes round k + S - 1: its stores have read it
      ptx::bulk_wait_read<1>();
      __syncthreads();
      issue(k + S - 1);
    }
  }
  ptx::bulk_wait_all();
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, int cluster, cudaStream_t stream) {
  static bool wide[64] = {};  // clusters of 16 allowed on the device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!wide[dev]) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    wide[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)((long long)a.batch * a.num_kv_heads * cluster);
  cfg.blockDim = kSelThreads;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
}

namespace {
cudaError_t compact_smem_limit(size_t smem) {
  static int smem_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (smem_set[dev] < (int)smem) {
    e = cudaFuncSetAttribute(evict_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    smem_set[dev] = (int)smem;
  }
  return cudaSuccess;
}
}  // namespace

cudaError_t occupancy_evict_compact(size_t smem, int* blocks_per_sm) {
  if (cudaError_t e = compact_smem_limit(smem)) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, evict_compact_kernel, kCompactThreads, smem);
}

cudaError_t launch_evict_compact(const CompactArgs& a, int grid, size_t smem, cudaStream_t stream) {
  if (cudaError_t e = compact_smem_limit(smem)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = (unsigned)grid;
  cfg.blockDim = kCompactThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.in_place ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_compact_kernel, a);
}

}  // namespace kvq
