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
// threshold and the first rows equal to it.  A digit whose matching keys are
// all kept ends the search (24 bits tell most weights apart).
//
// A cluster of CTAs holds one (sequence, kv head): each warp reads a
// contiguous stretch of the weights from global memory once and keeps it in
// registers, so the passes touch no memory but the histogram.  Weights of one
// head share a few exponents and may all be equal, so a histogram has a column
// per lane (bank = lane): no two lanes of a warp ever meet, whatever the
// values.  The columns' sums meet through the cluster's shared memory, where
// every CTA adds them up for itself: one cluster barrier a digit.  Integer
// adds: their order cannot show.
//
// Bound by instructions and the latency of the passes, not by HBM (4 bytes a
// row).  One 2048-bin histogram with its collisions took 118 us for 4 heads of
// 262,144 rows (1356 us for 512 heads of up to 131,072 rows); 12-bit digits in
// four copies 137 us, most of it in summing 4096 bins over 16 CTAs.

constexpr int kSelWarps = kSelThreads / 32;

// Ascending keys of ascending weights: -0 as +0, NaN (1) below everything; 0 is
// no row's.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  const uint32_t k = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return f == f ? k : 1u;
}

__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(const SelectArgs a) {
  __shared__ __align__(16) uint32_t hist[257 * 32];  // [bin][lane]; bin 256: keys that no longer match
  __shared__ uint32_t total[2][256];                 // this CTA's counts of a digit (two passes' worth)
  __shared__ uint32_t s_gt[kSelWarps], s_eq[kSelWarps], s_scan[8], s_digit[3], s_cta[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = (int)ptx::cluster_size(), rank = (int)ptx::cluster_rank();
  const int seg = (int)(blockIdx.x / (unsigned)cs);
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
    for (int i = rank * kSelThreads + tid; i < a.budget; i += cs * kSelThreads)
      keep[i] = i >= n ? -1 : (whole || i < a.sinks ? i : L - a.budget + i);
    return;
  }
  for (int i = rank * kSelThreads + tid; i < a.sinks + a.recent; i += cs * kSelThreads) {
    if (i < a.sinks) keep[i] = i;
    else keep[need_all + i] = L - a.recent + (i - a.sinks);
  }

  // The M rows between the ends, in runs of 32 from a multiple of 32 on (so
  // that a run meets one page, or two of 16 rows), go to as many CTAs as hold
  // them in registers, or to all of the cluster when SMs are free; the others
  // leave (a cluster barrier does not wait for CTAs that have left).
  const int M = L - a.sinks - a.recent;
  const int first = a.sinks & ~31;
  const int runs = (L - a.recent - first + 31) >> 5;
  constexpr int kHeld = kSelWarps * kSelKeys;  // runs that a CTA holds
  const int ctas = a.spread ? cs : min(cs, (runs + kHeld - 1) / kHeld);
  if (rank >= ctas) return;
  // this warp's runs: [r0, r0 + m), the warps in (CTA, warp) order
  const int per = (runs + ctas * kSelWarps - 1) / (ctas * kSelWarps);
  const int r0 = min(runs, (rank * kSelWarps + warp) * per);
  const int m = min(runs, r0 + per) - r0;
  const int pos0 = first + r0 * 32 + lane;  // this lane's row of run 0
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks_per_seq;
  const float* head = a.mass + ((size_t)h << a.log2_bs);
  const size_t page = (size_t)a.num_kv_heads << a.log2_bs;
  bool bad = false;
  // key of this lane's row of run j (0 outside the M rows); branch-free, so
  // that loads run ahead
  auto load = [&](int j) -> uint32_t {
    int pos = pos0 + j * 32;
    const bool in = (unsigned)(pos - a.sinks) < (unsigned)M;
    pos = in ? pos : a.sinks;
    const int id = bt[pos >> a.log2_bs];
    const bool fine = (unsigned)id < (unsigned)a.num_blocks;
    bad = bad || !fine;
    const uint32_t k = order_key(head[(fine ? (size_t)id : 0) * page + (pos & (a.block_size - 1))]);
    return in ? (fine ? k : 1u) : 0u;
  };
  // the first kSelKeys runs in registers, the rest read again in each pass
  uint32_t key[kSelKeys];
#pragma unroll
  for (int j0 = 0; j0 < kSelKeys; j0 += 8) {
#pragma unroll
    for (int j = j0; j < j0 + 8; ++j) key[j] = 0u;
    if (j0 < m) {
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) {
        const uint32_t k = load(min(j, m - 1));
        key[j] = j < m ? k : 0u;
      }
    }
  }
  // f(run, key) for this warp's runs; keys of 0 among them (rows outside the M,
  // runs past the last of a group of eight) are below every row's: they never
  // reach the threshold, whose digits are found from the top
  auto each = [&](auto f) {
#pragma unroll
    for (int j0 = 0; j0 < kSelKeys; j0 += 8) {
      if (j0 < m) {
#pragma unroll
        for (int j = j0; j < j0 + 8; ++j) f(j, key[j]);
      }
    }
    for (int j = kSelKeys; j < m; ++j) f(j, load(j));
  };

  uint32_t prefix = 0;
  int need = need_all;
  uint32_t T = 0;  // rows above it stay, and the first `need` equal to it
  uint32_t* my_hist = hist + lane;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256 * 32 / 4; i += kSelThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (pass == 0) {
      each([&](int, uint32_t k) { atomicAdd(&my_hist[(k >> 24) * 32], 1u); });
    } else {
      each([&](int, uint32_t k) {
        const uint32_t d = min((k >> shift) - (prefix << 8), 256u);
        atomicAdd(&my_hist[d * 32], 1u);
      });
    }
    __syncthreads();
    {
      // kSelThreads / 256 threads a bin, starting apart by bin so that a warp's
      // lanes read different banks
      constexpr int kPer = kSelThreads / 256, kCols = 32 / kPer;
      const int bin = tid / kPer, c0 = (tid % kPer) * kCols;
      uint32_t s = 0;
#pragma unroll
      for (int j = 0; j < kCols; ++j) s += hist[bin * 32 + c0 + ((j + bin) & (kCols - 1))];
#pragma unroll
      for (int o = 1; o < kPer; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tid % kPer == 0) total[pass & 1][bin] = s;
    }
    ptx::cluster_sync();
    // the cluster's counts, highest bin first, and the scan that finds the digit
    if (tid < 256) {
      const int bin = 255 - tid;
      const uint32_t at = ptx::smem_u32(&total[pass & 1][bin]);
      uint32_t cnt = 0;
      for (int r = 0; r < ctas; r += 4) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = r + j < ctas ? ptx::ld_cluster_u32(at, (uint32_t)(r + j)) : 0u;
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
        s_digit[2] = cnt;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | s_digit[0];
    need -= (int)s_digit[1];
    T = prefix << shift;
    if ((int)s_digit[2] == need && T > 0) {
      // every key with this prefix stays (none of them at 0: then all M would)
      T -= 1;
      need = 0;
      break;
    }
  }
  if (bad) atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);

  // ---- ordered output
  uint32_t gt = 0, eq = 0;
  each([&](int, uint32_t k) {
    gt += k > T;
    eq += k == T;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
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
  if (lane < rank) {
    bg = ptx::ld_cluster_u32(ptx::smem_u32(&s_cta[0]), (uint32_t)lane);
    be = ptx::ld_cluster_u32(ptx::smem_u32(&s_cta[1]), (uint32_t)lane);
  }
  if (lane < warp) {
    bg += s_gt[lane];
    be += s_eq[lane];
  }
  bg = __reduce_add_sync(0xffffffffu, bg);
  be = __reduce_add_sync(0xffffffffu, be);
  const uint32_t below = (1u << lane) - 1u;
  int32_t* mid = keep + a.sinks;
  if (need == 0) {
    each([&](int j, uint32_t k) {
      const uint32_t mg = __ballot_sync(0xffffffffu, k > T);
      if (k > T) mid[bg + __popc(mg & below)] = pos0 + j * 32;
      bg += __popc(mg);
    });
  } else {
    each([&](int j, uint32_t k) {
      const uint32_t mg = __ballot_sync(0xffffffffu, k > T), me = __ballot_sync(0xffffffffu, k == T);
      const uint32_t g = bg + __popc(mg & below), e = be + __popc(me & below);
      if (k > T || (k == T && e < (uint32_t)need)) mid[g + min(e, (uint32_t)need)] = pos0 + j * 32;
      bg += __popc(mg);
      be += __popc(me);
    });
  }
  ptx::cluster_sync();  // no CTA leaves while another reads its counts
}

// ----------------------------------------------------------------- compact
//
// Row i of a (sequence, kv head) becomes row keep[i] >= i (ascending): a
// gather of rows of Dp bytes and a dense, page-wise store, so bound by HBM
// (kept rows read once, written once).  The units are `rows` consecutive
// destination rows of one (sequence, kv head); a CTA takes units grid apart,
// one a round, through a ring of shared-memory stages.
//
// In place, a unit's destination rows may hold rows that its own or an earlier
// unit of the same (sequence, kv head) has yet to read -- never a later one's,
// whose sources lie at or behind its own destination.  Units are numbered so
// that earlier chunks come in the same or an earlier round; a round's stores
// therefore wait until every CTA has loaded its unit of that round (a counter
// per round, all CTAs resident: a cooperative launch).  The loads of later
// rounds need no wait, so they are in flight meanwhile.  Every wait is bounded.
//
// Roles, so that no latency of a round stands behind another's (with one group
// of threads doing all of it in turn, 4 heads of 131,072 kept rows of 520
// bytes took 197 us; with the look-ups in the loading warps 119):
//   warps 0-3   load: 16-byte cp.async per chunk of a row, 4-byte ones for the
//               scales and weights
//   warps 4-7   store: shared memory -> destination pages
//   warps 8-11  look up the kept rows and pages of the units ahead
//   warp 12     reports this CTA's loaded rounds
//   warp 13     waits for a round's reports and lets the stores go
constexpr int kRole = 128;    // threads of a loading, storing or looking-up role
constexpr int kLookAhead = 8; // units looked up ahead

__global__ void __launch_bounds__(kCompactThreads) evict_compact_kernel(const CompactArgs a) {
  extern __shared__ __align__(128) uint8_t cmp_smem[];
  // looked-up units, by round mod kLookAhead: cache slots (block * block size
  // + row) of the rows' sources and destinations, -1: none
  __shared__ int s_src[kLookAhead][kCompactRows], s_dst[kLookAhead][kCompactRows];
  __shared__ int s_n[kLookAhead], s_h[kLookAhead];  // rows to move (0: none), kv head
  __shared__ __align__(8) uint64_t look_full[kLookAhead], look_empty[kLookAhead];
  __shared__ __align__(8) uint64_t full[kCompactStages], empty[kCompactStages], go[kCompactStages];
  __shared__ int s_stop;  // a wait gave up: nothing is stored from there on
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = a.stages;
  if (tid == 0) {
    for (int q = 0; q < kLookAhead; ++q) {
      ptx::mbar_init(&look_full[q], kRole);
      ptx::mbar_init(&look_empty[q], kRole / 32);
    }
    for (int s = 0; s < S; ++s) {
      // a loader arrives twice: itself, and behind its copies
      ptx::mbar_init(&full[s], 2 * kRole);
      ptx::mbar_init(&empty[s], kRole / 32);
      ptx::mbar_init(&go[s], 1);
    }
    ptx::fence_mbar_init();
    s_stop = 0;
  }
  __syncthreads();
  ptx::griddep_wait();
  const int segs = a.batch * a.num_kv_heads;
  const int rounds = (a.units + (int)gridDim.x - 1) / (int)gridDim.x;
  const int code_bytes = a.rows * a.row_bytes;  // one side of a stage
  const int nf = a.n_scale[0] + a.n_scale[1] + (a.mass ? 1 : 0);
  const int row_chunks = a.row_bytes / 16, unit_chunks = row_chunks * a.sides;  // 16-byte chunks of a row, of both sides
  volatile int* stop = &s_stop;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!*stop && !ptx::mbar_wait_bounded(bar, (uint32_t)phase & 1u)) {
      atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
      *stop = 1;
    }
  };
  // [block, kv head, row] index of a cache slot
  auto row_at = [&](int slot, int h) -> size_t {
    return (((size_t)(slot >> a.log2_bs) * a.num_kv_heads + h) << a.log2_bs) + (slot & (a.block_size - 1));
  };
  // f(row, side, byte offset in the side's row) for this thread's 16-byte
  // chunks of an n-row unit (t of kRole threads)
  auto chunks = [&](int t, int n, auto f) {
    const int dr = kRole / unit_chunks, dc = kRole - dr * unit_chunks;
    int r = t / unit_chunks, c = t - r * unit_chunks;
    while (r < n) {
      const int side = c >= row_chunks ? 1 : 0;
      f(r, side, (c - side * row_chunks) * 16);
      r += dr;
      c += dc;
      if (c >= unit_chunks) {
        c -= unit_chunks;
        ++r;
      }
    }
  };

  if (warp < 4) {
    // ============================================================== loaders
    for (int k = 0; k < rounds; ++k) {
      const int s = k % S, q = k % kLookAhead;
      uint8_t* st = cmp_smem + (size_t)s * a.stage_bytes;
      wait(&look_full[q], k / kLookAhead);
      if (k >= S) wait(&empty[s], k / S - 1);
      const int n = *stop ? 0 : s_n[q], h = s_h[q];
      chunks(tid, n, [&](int r, int side, int off) {
        const int slot = s_src[q][r];
        if (slot >= 0)
          ptx::cp_async16(st + side * code_bytes + r * a.row_bytes + off,
                          a.codes[side] + row_at(slot, h) * a.row_bytes + off);
      });
      if (tid < n && nf > 0 && s_src[q][tid] >= 0) {
        const size_t row = row_at(s_src[q][tid], h);
        float* f = reinterpret_cast<float*>(st + a.sides * code_bytes) + tid;
        for (int side = 0; side < a.sides; ++side)
          for (int j = 0; j < a.n_scale[side]; ++j, f += a.rows)
            ptx::cp_async4(f, a.scale[side] + row * a.n_scale[side] + j);
        if (a.mass) ptx::cp_async4(f, a.mass + row);
      }
      ptx::cp_async_arrive(&full[s]);
      ptx::mbar_arrive(&full[s]);
    }
  } else if (warp < 8) {
    // ============================================================== storers
    const int t = tid - kRole;
    for (int k = 0; k < rounds; ++k) {
      const int s = k % S, q = k % kLookAhead;
      const uint8_t* st = cmp_smem + (size_t)s * a.stage_bytes;
      wait(&full[s], k / S);
      if (a.in_place) wait(&go[s], k / S);
      const int n = *stop ? 0 : s_n[q], h = s_h[q];
      chunks(t, n, [&](int r, int side, int off) {
        const uint4 v = *reinterpret_cast<const uint4*>(st + side * code_bytes + r * a.row_bytes + off);
        const int slot = s_dst[q][r];
        if (slot >= 0) *reinterpret_cast<uint4*>(a.codes[side] + row_at(slot, h) * a.row_bytes + off) = v;
      });
      if (t < n && nf > 0 && s_dst[q][t] >= 0) {
        const size_t row = row_at(s_dst[q][t], h);
        const float* f = reinterpret_cast<const float*>(st + a.sides * code_bytes) + t;
        for (int side = 0; side < a.sides; ++side)
          for (int j = 0; j < a.n_scale[side]; ++j, f += a.rows) a.scale[side][row * a.n_scale[side] + j] = *f;
        if (a.mass) a.mass[row] = *f;
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&empty[s]);
        ptx::mbar_arrive(&look_empty[q]);
      }
    }
  } else if (warp < 12) {
    // ============================================================= look-ups
    const int r = tid - 2 * kRole;
    const int cap = a.max_blocks_per_seq << a.log2_bs;
    auto slot_of = [&](const int32_t* table, int b, int p) -> int {
      const int id = table[(size_t)b * a.max_blocks_per_seq + (p >> a.log2_bs)];
      if (id < 0 || id >= a.num_blocks) {
        atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
        return -1;
      }
      return (id << a.log2_bs) + (p & (a.block_size - 1));
    };
    for (int k = 0; k < rounds; ++k) {
      const int q = k % kLookAhead;
      if (k >= kLookAhead) wait(&look_empty[q], k / kLookAhead - 1);
      // unit of round k: chunk-major over the (sequence, kv head) pairs
      const long long u = (long long)k * gridDim.x + blockIdx.x;
      int n = 0, h = 0;
      if (u < a.units) {
        const int chunk = (int)(u / segs), seg = (int)(u - (long long)chunk * segs);
        const int b = seg / a.num_kv_heads, i = (chunk << a.log2_rows) + r;
        h = seg - b * a.num_kv_heads;
        // (both loads at once: entries of keep behind the kept ones are there)
        const int p = r < a.rows && i < a.budget ? a.keep[(size_t)seg * a.budget + i] : -1;
        n = min(a.rows, min(a.kept_lens[b], a.budget) - (chunk << a.log2_rows));
        if (r < n) {
          int src = -1;
          // (in place, a row from before its destination may be gone)
          if (p < (a.in_place ? i : 0) || p >= cap) atomicOr(a.err, KVQ_DEVERR_KEEP_INDEX);
          else src = slot_of(a.block_table, b, p);
          s_src[q][r] = src;
          // (budget <= capacity: i is inside the table)
          s_dst[q][r] = src >= 0 ? slot_of(a.dst_table, b, i) : -1;
          if (r == n - 1) {
            // ascending rows whose last is in its place all are
            s_n[q] = a.in_place && p == i ? 0 : n;
            s_h[q] = h;
          }
        }
      }
      if (n <= 0 && r == 0) s_n[q] = 0;
      ptx::mbar_arrive(&look_full[q]);
    }
  } else if (a.in_place && lane == 0) {
    for (int k = 0; k < rounds; ++k) {
      const int s = k % S;
      if (warp == 12) {
        // ======================================================== reporter
        // (the copies' completion is observed through the barrier; the add
        // releases it to whoever reads the full count)
        wait(&full[s], k / S);
        ptx::red_release_add(&a.round_count[k], 1u);
      } else {
        // ========================================================== poller
        // Round k's count is full only once this CTA has loaded its own unit,
        // hence freed the stage of round k - S: `go` is never a phase ahead.
        const uint64_t t0 = ptx::globaltimer_ns();
        uint32_t i = 0;
        while (!*stop && ptx::ld_acquire(&a.round_count[k]) < gridDim.x) {
          if ((++i & 63u) == 0u && ptx::globaltimer_ns() - t0 > ptx::kWaitLimitNs) {
            atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
            *stop = 1;
          }
        }
        ptx::mbar_arrive(&go[s]);
      }
    }
  }
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
  static std::atomic<int> smem_set[64];
  return raise_smem_limit(reinterpret_cast<const void*>(evict_compact_kernel), smem_set, smem);
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
