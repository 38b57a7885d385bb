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
// four copies 137 us, most of it in summing 4096 bins over 16 CTAs; a list of
// the keys with the threshold's upper half in place of the last two digits
// gained nothing (276 against 282 us).

constexpr int kSelWarps = kSelThreads / 32;

// Ascending keys of ascending weights: -0 as +0, NaN (1) below everything; 0 is
// no row's.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  const uint32_t k = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return f == f ? k : 1u;
}

// What both kernels begin with: the lengths, and the rows that stay whatever
// their weight (t of `threads` threads of the head).  False: there are no
// others to choose.
struct SelectHead {
  int L, need;  // rows, and how many of those between the ends stay
};
__device__ __forceinline__ bool select_ends(const SelectArgs& a, int b, int h, int t, int threads, SelectHead& hd) {
  const int raw = a.seq_lens[b];
  const int L = raw < 0 ? 0 : (raw > a.lim ? a.lim : raw);
  if (raw != L && h == 0 && t == 0) atomicOr(a.err, KVQ_DEVERR_SEQ_LEN);
  int32_t* keep = a.keep + (size_t)(b * a.num_kv_heads + h) * a.budget;
  const int n = min(L, a.budget);
  if (h == 0 && t == 0) a.kept_lens[b] = n;
  // everything stays, or only the protected ends do
  const int need = a.budget - a.sinks - a.recent;
  const bool whole = L <= a.budget;
  if (whole || need == 0) {
    for (int i = t; i < a.budget; i += threads) keep[i] = i >= n ? -1 : (whole || i < a.sinks ? i : L - a.budget + i);
    return false;
  }
  for (int i = t; i < a.sinks + a.recent; i += threads) {
    if (i < a.sinks) keep[i] = i;
    else keep[need + i] = L - a.recent + (i - a.sinks);
  }
  hd.L = L;
  hd.need = need;
  return true;
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

  SelectHead hd;
  if (!select_ends(a, b, h, rank * kSelThreads + tid, cs * kSelThreads, hd)) return;  // (the whole cluster)
  const int L = hd.L;
  int32_t* keep = a.keep + (size_t)seg * a.budget;

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
  auto each_held = [&](auto f) {
#pragma unroll
    for (int j0 = 0; j0 < kSelKeys; j0 += 8) {
      if (j0 < m) {
#pragma unroll
        for (int j = j0; j < j0 + 8; ++j) f(j, key[j]);
      }
    }
  };
  auto each = [&](auto f) {
    each_held(f);
    for (int j = kSelKeys; j < m; ++j) f(j, load(j));
  };

  uint32_t prefix = 0;
  int need = hd.need;
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
  // Runs that are read again may give other weights in each pass, when another
  // stream writes them meanwhile: then more than a.need rows may have been
  // counted, or `need` have gone below 0.  A warp whose rows would end past the
  // head's places writes none, and the runs that are read once more are bounded
  // store by store (all of them so: 6% of a call whose rows are all held).
  if (bg + gt + min(be + eq, (uint32_t)need) <= (uint32_t)a.need) {
    if (need == 0) {
      each_held([&](int j, uint32_t k) {
        const uint32_t mg = __ballot_sync(0xffffffffu, k > T);
        if (k > T) mid[bg + __popc(mg & below)] = pos0 + j * 32;
        bg += __popc(mg);
      });
    } else {
      each_held([&](int j, uint32_t k) {
        const uint32_t mg = __ballot_sync(0xffffffffu, k > T), me = __ballot_sync(0xffffffffu, k == T);
        const uint32_t g = bg + __popc(mg & below), e = be + __popc(me & below);
        if (k > T || (k == T && e < (uint32_t)need)) mid[g + min(e, (uint32_t)need)] = pos0 + j * 32;
        bg += __popc(mg);
        be += __popc(me);
      });
    }
#pragma unroll 8
    for (int j = kSelKeys; j < m; ++j) {
      const uint32_t k = load(j), mg = __ballot_sync(0xffffffffu, k > T), me = __ballot_sync(0xffffffffu, k == T);
      const uint32_t e = be + __popc(me & below), to = bg + __popc(mg & below) + min(e, (uint32_t)need);
      if ((k > T || (k == T && e < (uint32_t)need)) && to < (uint32_t)a.need) mid[to] = pos0 + j * 32;
      bg += __popc(mg);
      be += __popc(me);
    }
  }
  ptx::cluster_sync();  // no CTA leaves while another reads its counts
}

// -------------------------------------------------------- select, many heads
//
// With enough long heads (the rule is with the launch) one CTA takes a head and
// reads its weights once:
//   1. a sample of 4096 rows, evenly spread, brackets the threshold: two ranks
//      five standard deviations to either side of the wanted one, to 16 bits;
//   2. one pass over the weights (16 bytes a lane) marks the rows above the
//      bracket and those inside it, a bit each: two compares and two votes a
//      row, nothing else;
//   3. the weights of the rows inside are read again into a list, whose radix
//      select by key and then by row (the lower row first), digits of 8 bits,
//      adds its rows to the bits of the rows above;
//   4. the bits give the rows in order.
// Exact whatever the sample was: when the wanted rank turns out not to lie in
// the bracket, or the list overflows (thousands of rows of nearly the same
// weight, as exact zeros under a steep bias), the head goes through the digits
// of the kernel above, reading its weights again for each (from L2): with 98% of
// the weights equal 512 heads take 404 us (the clusters 280), 80 heads of 131,072
// rows 257 (68), which the host cannot know.  512 heads of up to 131,072 rows: 106 us
// (276 with the clusters above, whose loads, digit passes, counts and output
// took 107, 62, 70 and 38 us of it).  304 heads of 131,072 rows take 89: 25 the
// sample's scattered reads and digits, 33 the pass (4.8 TB/s), 15 the list and
// its digits, the rest launch and output.  Half the sample misses the bracket
// often enough to lose what it saves.
constexpr int kManyThreads = kSelThreads, kManyWarps = kManyThreads / 32;
constexpr int kManySample = 8;                              // samples a thread
constexpr int kManySamples = kManySample * kManyThreads;
static_assert(2 * kManyList >= 257 * 32, "the digits' columns take the list's place");

// The digit of the need-th largest key from a digit's counts (every warp for
// itself, eight bins a lane from the highest on).
__device__ __forceinline__ void find_digit(const uint32_t* bins, uint32_t need, int lane, uint32_t& digit,
                                           uint32_t& same, uint32_t& before) {
  uint32_t cnt[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += cnt[i] = bins[255 - (8 * lane + i)];
  uint32_t above = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
    if (lane >= o) above += y;
  }
  const int owner = max(0, __ffs(__ballot_sync(0xffffffffu, above >= need)) - 1);
  above -= sum;
  uint32_t d = 0, c = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!found) {
      if (above + cnt[i] >= need) {
        found = true;
        d = 255u - (8 * lane + i);
        c = cnt[i];
      } else {
        above += cnt[i];
      }
    }
  }
  digit = __shfl_sync(0xffffffffu, d, owner);
  same = __shfl_sync(0xffffffffu, c, owner);
  before = __shfl_sync(0xffffffffu, above, owner);
}

__global__ void __launch_bounds__(kManyThreads, 2) evict_select_many_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint32_t many_smem[];
  uint32_t* lkey = many_smem;         // [kManyList] keys inside the bracket, less its lower end
  uint32_t* lrow = lkey + kManyList;  // [kManyList] their rows, from `first` on
  uint32_t* hist = many_smem;         // [257][32] a digit's counts, a column a lane
  // [blocks][2][4] a block of 128 rows: the rows that stay, then those inside
  // the bracket; bit l of word c is row 4 l + c
  uint32_t* mask = lrow + kManyList;
  __shared__ uint32_t bins[2][256];
  __shared__ uint32_t s_list, s_above, s_valid, s_warp[kManyWarps], s_equal[kManyWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // the longest sequences first: the heads that start last end the call
  // (64 sequences of up to 131,072 rows: 115 against 134 us)
  const int nth = (int)blockIdx.x / a.num_kv_heads, h = (int)blockIdx.x - nth * a.num_kv_heads;
  if (a.batch <= 128) {
    int* lens = reinterpret_cast<int*>(bins[0]);
    const int len = tid < a.batch ? a.seq_lens[tid] : 0;
    if (tid < a.batch) lens[tid] = len;
    __syncthreads();
    if (tid < a.batch) {
      int ahead = 0;
#pragma unroll 4
      for (int i = 0; i < a.batch; ++i) ahead += lens[i] > len || (lens[i] == len && i < tid);
      if (ahead == nth) s_list = (uint32_t)tid;
    }
  } else if (tid == 0) {
    s_list = (uint32_t)nth;
  }
  __syncthreads();
  const int b = (int)s_list, seg = b * a.num_kv_heads + h;
  __syncthreads();
  SelectHead hd;
  if (!select_ends(a, b, h, tid, kManyThreads, hd)) return;
  const int L = hd.L;
  const int M = L - a.sinks - a.recent, first = a.sinks & ~31, runs = (L - a.recent - first + 31) >> 5;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks_per_seq;
  const char* head = reinterpret_cast<const char*>(a.mass + ((size_t)h << a.log2_bs));
  const uint32_t page_bytes = 4u * ((uint32_t)a.num_kv_heads << a.log2_bs);  // (the host's check: below 2^32)
  const bool two = a.log2_bs == 4;  // a run of 32 rows lies on one page, or on two of 16 rows
  bool bad = false;
  if (tid == 0) s_list = s_above = s_valid = 0;

  // the page of run base + lane (of half a run, when two), -1: unreadable or none
  auto look_up = [&](int base) -> int {
    const int x = two ? 16 * lane : 32 * lane;
    if (lane >= (two ? 16 : 8) || first + base * 32 + x >= L - a.recent) return -1;
    const int id = bt[(first + base * 32 + x) >> a.log2_bs];
    if ((unsigned)id < (unsigned)a.num_blocks) return id;
    bad = true;
    return -1;
  };
  // this lane's weights of the eight runs from base on
  auto fetch = [&](int base, int ids, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int id = __shfl_sync(0xffffffffu, ids, two ? 2 * i + (lane >> 4) : i);
      f[i] = __uint_as_float(0x7FC00000u);
      if (id >= 0)
        f[i] = *reinterpret_cast<const float*>(head + (uint64_t)(uint32_t)id * page_bytes +
                                               4u * (uint32_t)((first + 32 * (base + i) + lane) & (a.block_size - 1)));
    }
  };
  // f(run, key) for the runs of [r0, r1), eight at a time from r0 on, `step`
  // apart; key 0: not one of the M rows
  auto rows = [&](int r0, int r1, int step, auto f) {
    if (r0 >= r1) return;
    float now[8], next[8];
    fetch(r0, look_up(r0), now);
    int ids = look_up(r0 + step);
    for (int base = r0; base < r1; base += step) {
      fetch(base + step, ids, next);
      ids = look_up(base + 2 * step);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = (unsigned)(first + 32 * (base + i) + lane - a.sinks) < (unsigned)M && base + i < r1;
        f(base, i, in ? order_key(now[i]) : 0u);
        now[i] = next[i];
      }
    }
  };
  // one digit of the need-th largest of the keys that `each` goes through
  uint32_t* my_hist = hist + lane;
  auto digit_of = [&](auto each, int shift, uint32_t prefix, uint32_t need, uint32_t& digit, uint32_t& same,
                      uint32_t& before) {
    __syncthreads();
    for (int i = tid; i < 256 * 32 / 4; i += kManyThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    each([&](uint32_t k) {
      const uint32_t d = shift == 24 ? k >> 24 : min((k >> shift) - (prefix << 8), 256u);
      atomicAdd(&my_hist[d * 32], 1u);
    });
    __syncthreads();
    const int bin = tid >> 1, c0 = (tid & 1) * 16;  // two threads a bin
    uint32_t s = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) s += hist[bin * 32 + c0 + ((j + bin) & 15)];
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    if ((tid & 1) == 0) bins[0][bin] = s;
    __syncthreads();
    find_digit(bins[0], need, lane, digit, same, before);
  };

  // key of row `row` from `first` on
  auto key_at = [&](int row) -> uint32_t {
    const int pos = first + row, id = bt[pos >> a.log2_bs];
    if ((unsigned)id >= (unsigned)a.num_blocks) return 1u;
    return order_key(*reinterpret_cast<const float*>(head + (uint64_t)(uint32_t)id * page_bytes +
                                                     4u * (uint32_t)(pos & (a.block_size - 1))));
  };

  // ---- the bracket [lo, hi]
  uint32_t need = (uint32_t)hd.need, lo = 1u, hi = 0xFFFFFFFFu;
  if (M > kManyList) {
    uint32_t smp[kManySample];
#pragma unroll
    for (int j = 0; j < kManySample; ++j) {
      smp[j] = key_at(a.sinks - first + (int)(((long long)(tid + j * kManyThreads) * M) / kManySamples));
    }
    auto each = [&](auto f) {
#pragma unroll
      for (int j = 0; j < kManySample; ++j) f(smp[j]);
    };
    const float r = (float)need / (float)M * kManySamples;
    // five standard deviations to either side (one head in a million misses),
    // fewer if the list would not hold them
    const float sigma = sqrtf(r * fmaxf(0.0f, 1.0f - r / kManySamples));
    const float half = fminf(5.0f * sigma + 2.0f, 0.45f * kManyList * kManySamples / (float)M);
    const int rank_hi = (int)floorf(r - half), rank_lo = (int)ceilf(r + half);
    uint32_t d, d2, same, before, e, before_lo;
    digit_of(each, 24, 0u, (uint32_t)max(1, rank_hi), d, same, before);
    find_digit(bins[0], (uint32_t)min(kManySamples, rank_lo), lane, e, same, before_lo);
    if (rank_hi >= 1) {
      digit_of(each, 16, d, (uint32_t)rank_hi - before, d2, same, before);
      hi = (d << 24) | (d2 << 16) | 0xFFFFu;
    }
    if (rank_lo <= kManySamples) {
      digit_of(each, 16, e, (uint32_t)rank_lo - before_lo, d2, same, before);
      lo = max(1u, (e << 24) | (d2 << 16));
    }
  }
  __syncthreads();

  // ---- the pass over the weights.  Floats compare as their keys do, but for
  // the two zeros and NaN, which the list's exact keys put right: a row above
  // as a float is above, and a row neither above nor below the lower end is
  // looked at again.
  const int blocks = (L - a.recent - first + 127) >> 7;
  {
    auto value = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); };
    const float lo_f = value(lo), hi_f = value(hi);
    constexpr int kStep = kManyWarps * 4;  // four blocks a warp at a time
    // the page of the 16 rows from base * 128 + 16 * lane on, -1: unreadable or none
    auto look_up16 = [&](int base) -> int {
      const int pos = first + base * 128 + 16 * lane;
      if (pos >= L - a.recent) return -1;
      const int id = bt[pos >> a.log2_bs];
      if ((unsigned)id < (unsigned)a.num_blocks) return id;
      bad = true;
      return -1;
    };
    auto fetch4 = [&](int base, int ids, float4 (&f)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int id = __shfl_sync(0xffffffffu, ids, 8 * i + (lane >> 2));
        const float nan = __uint_as_float(0x7FC00000u);
        f[i] = make_float4(nan, nan, nan, nan);
        if (id >= 0)
          f[i] = *reinterpret_cast<const float4*>(
              head + (uint64_t)(uint32_t)id * page_bytes +
              4u * (uint32_t)((first + 128 * (base + i) + 4 * lane) & (a.block_size - 1)));
      }
    };
    float4 now[4], next[4];
    int ids = look_up16(warp * 4);
    if (warp * 4 < blocks) fetch4(warp * 4, ids, now);
    ids = look_up16(warp * 4 + kStep);
    for (int base = warp * 4; base < blocks; base += kStep) {
      fetch4(base + kStep, ids, next);
      ids = look_up16(base + 2 * kStep);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
        uint32_t word = 0;
        const int row0 = first + 128 * (base + i);
        const bool inner = row0 >= a.sinks && row0 + 128 <= L - a.recent;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool ok = inner || (unsigned)(row0 + 4 * lane + c - a.sinks) < (unsigned)M;
          const uint32_t up = __ballot_sync(0xffffffffu, ok && x[c] > hi_f);
          const uint32_t in = __ballot_sync(0xffffffffu, ok && !(x[c] > hi_f) && !(x[c] < lo_f));
          if (lane == c) word = up;
          if (lane == 4 + c) word = in;
        }
        if (lane < 8 && base + i < blocks) mask[(base + i) * 8 + lane] = word;
        now[i] = next[i];
      }
    }
  }
  __syncthreads();

  // ---- the list: the rows, then their keys
  {
    uint32_t above = 0, mine = 0;
    for (int w = tid; w < blocks * 4; w += kManyThreads) {
      above += __popc(mask[(w >> 2) * 8 + (w & 3)]);
      mine += __popc(mask[(w >> 2) * 8 + 4 + (w & 3)]);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    uint32_t at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    uint32_t start = 0;
    if (lane == 31) {
      start = atomicAdd(&s_list, at);
      atomicAdd(&s_above, above);
    }
    at += __shfl_sync(0xffffffffu, start, 31) - mine;
    for (int w = tid; w < blocks * 4; w += kManyThreads) {
      for (uint32_t m = mask[(w >> 2) * 8 + 4 + (w & 3)]; m; m &= m - 1, ++at)
        if (at < kManyList) lrow[at] = (uint32_t)((w >> 2) * 128 + 4 * (__ffs(m) - 1) + (w & 3));
    }
  }
  if (tid < 256) bins[0][tid] = 0;
  __syncthreads();
  const uint32_t n = s_list;
  if (n <= kManyList) {
    uint32_t above = 0, valid = 0;
#pragma unroll 4
    for (uint32_t i = tid; i < n; i += kManyThreads) {
      const uint32_t row = lrow[i], k = key_at((int)row);
      if (k > hi) {
        atomicOr(&mask[(row >> 7) * 8 + (row & 3u)], 1u << ((row & 127u) >> 2));
        ++above;
      }
      const bool in = k - lo <= hi - lo;
      valid += in;
      lkey[i] = in ? k - lo : 0u;
      if (!in) lrow[i] = 0xFFFFFFFFu;  // not one of the list's: below every entry
    }
    above = __reduce_add_sync(0xffffffffu, above);
    valid = __reduce_add_sync(0xffffffffu, valid);
    if (lane == 0) {
      atomicAdd(&s_above, above);
      atomicAdd(&s_valid, valid);
    }
  }
  __syncthreads();
  int32_t* mid = a.keep + (size_t)seg * a.budget + a.sinks;
  if (n <= kManyList && s_above <= need && need - s_above <= s_valid) {
    // ---- its need-th largest, the lowest row among equals
    need -= s_above;
    auto entry = [&](uint32_t i) { return ((uint64_t)lkey[i] << 32) | (uint32_t)~lrow[i]; };
    int shift = 64 - __clz((int)((hi - lo) | 1u));  // no entry has bits above
    uint64_t pre = 0;                               // the entries of pre at `shift` and above it stay
    const bool none = need == 0, all = need == s_valid;
    bool open = !none && !all;
    for (int pass = 0; open && shift > 0; ++pass) {
      const int width = min(8, shift), low = shift - width;
      uint32_t* cnt = bins[pass & 1];
      if (tid < 256) bins[(pass + 1) & 1][tid] = 0;
      for (uint32_t i = tid; i < n; i += kManyThreads) {
        const uint64_t e = entry(i);
        if (pass == 0 || (e >> shift) == pre) atomicAdd(&cnt[(uint32_t)(e >> low) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      uint32_t d, same, before;
      find_digit(cnt, need, lane, d, same, before);
      pre = (pre << width) | d;
      need -= before;
      shift = low;
      open = same > need;
      __syncthreads();
    }
    if (!none) {
      for (uint32_t i = tid; i < n; i += kManyThreads) {
        const uint32_t row = lrow[i];
        if (row != 0xFFFFFFFFu && (all || (entry(i) >> shift) >= pre))
          atomicOr(&mask[(row >> 7) * 8 + (row & 3u)], 1u << ((row & 127u) >> 2));
      }
    }
    __syncthreads();

    // ---- the rows in order, a stretch of blocks a warp
    const int per = (blocks + kManyWarps - 1) / kManyWarps, w0 = min(blocks, warp * per), w1 = min(blocks, w0 + per);
    uint32_t kept = 0;
    for (int w = 4 * w0 + lane; w < 4 * w1; w += 32) kept += __popc(mask[(w >> 2) * 8 + (w & 3)]);
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0) s_warp[warp] = kept;
    __syncthreads();
    uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    if (hd.need <= 2 * kManyList && hd.need <= M / 16) {
      // few of them: a block a lane, through shared memory in the list's place
      // (304 heads of 131,072 rows, 4096 kept: 89 against 100 us with the
      // stores of a lane or two each below; of 32,768 rows, 4096 kept 38
      // against 37, 12,000 kept 41 against 35)
      uint32_t* stage = many_smem;
      for (int g = w0; g < w1; g += 32) {
        uint4 m = make_uint4(0, 0, 0, 0);
        if (g + lane < w1) m = *reinterpret_cast<const uint4*>(mask + (g + lane) * 8);
        const uint32_t mine = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
        uint32_t to = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, to, o);
          if (lane >= o) to += y;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, to, 31);
        to += at - mine;
        at += total;
        for (uint32_t some = m.x | m.y | m.z | m.w; some; some &= some - 1) {
          const int l = __ffs(some) - 1;
          const uint32_t four = (m.x >> l & 1u) | (m.y >> l & 1u) << 1 | (m.z >> l & 1u) << 2 | (m.w >> l & 1u) << 3;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (four >> c & 1u) {
              if (to < 2 * kManyList) stage[to] = (uint32_t)(first + 128 * (g + lane) + 4 * l + c);
              ++to;
            }
        }
      }
      __syncthreads();
      for (int i = tid; i < hd.need; i += kManyThreads) mid[i] = (int)stage[i];
      if (bad) atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
      return;
    }
    // four blocks at a time: how many of each block's rows the lanes below
    // have, a byte a block (128 at most), from one scan
    for (int g = w0; g < w1; g += 4) {
      uint32_t nib[4], mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 m = make_uint4(0, 0, 0, 0);
        if (g + i < w1) m = *reinterpret_cast<const uint4*>(mask + (g + i) * 8);
        const uint32_t x = m.x >> lane & 1u, y = m.y >> lane & 1u, z = m.z >> lane & 1u, v = m.w >> lane & 1u;
        nib[i] = x | y << 1 | z << 2 | v << 3;
        mine |= (x + y + z + v) << (8 * i);
      }
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t total = __shfl_sync(0xffffffffu, incl, 31), below = incl - mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t to = at + (below >> (8 * i) & 255u);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (nib[i] >> c & 1u) {
            // (never more than that, unless another stream changes the weights meanwhile)
            if (to < (uint32_t)hd.need) mid[to] = first + 128 * (g + i) + 4 * lane + c;
            ++to;
          }
        at += total >> (8 * i) & 255u;
      }
    }
  } else {
    // ---- digit by digit over all rows
    auto each = [&](auto f) { rows(warp * 8, runs, kManyWarps * 8, [&](int, int, uint32_t k) { f(k); }); };
    uint32_t T = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      uint32_t d, same, before;
      digit_of(each, 24 - 8 * pass, T, need, d, same, before);
      T = (T << 8) | d;
      need -= before;
    }
    // the rows above T, and the first `need` equal to it, a stretch of runs a warp
    const int per = (runs + kManyWarps - 1) / kManyWarps, w0 = min(runs, warp * per), w1 = min(runs, w0 + per);
    uint32_t gt = 0, eq = 0;
    rows(w0, w1, 8, [&](int, int, uint32_t k) {
      gt += k > T;
      eq += k == T;
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      s_warp[warp] = gt;
      s_equal[warp] = eq;
    }
    __syncthreads();
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? s_equal[lane] : 0u);
    const uint32_t below = (1u << lane) - 1u;
    rows(w0, w1, 8, [&](int base, int i, uint32_t k) {
      const uint32_t up = __ballot_sync(0xffffffffu, k > T), same = __ballot_sync(0xffffffffu, k == T);
      const uint32_t e = eq + __popc(same & below), to = gt + __popc(up & below) + min(e, need);
      if ((k > T || (k == T && e < need)) && to < (uint32_t)hd.need) mid[to] = first + (base + i) * 32 + lane;
      gt += __popc(up);
      eq += __popc(same);
    });
  }
  if (bad) atomicOr(a.err, KVQ_DEVERR_BLOCK_ID);
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
  static std::atomic<bool> wide[64];  // clusters of 16 allowed on the device (host threads may set it side by side)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!wide[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    wide[dev].store(true, std::memory_order_release);
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

size_t select_many_smem(int rows) { return (size_t)(2 * kManyList + 8 * ((rows + 127) / 128 + 1)) * 4; }

cudaError_t launch_evict_select_many(const SelectArgs& a, cudaStream_t stream) {
  static std::atomic<int> smem_set[64];
  const size_t smem = select_many_smem(a.lim);
  if (cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(evict_select_many_kernel), smem_set, smem)) return e;
  return launch_pdl(evict_select_many_kernel, (unsigned)(a.batch * a.num_kv_heads), kManyThreads, smem, stream, a);
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
