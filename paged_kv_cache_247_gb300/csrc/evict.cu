// Eviction from the paged cache: which positions a sequence keeps
// (kv_evict_select) and the move of their rows to the front (kv_compact).
//
// A sequence keeps a bounded cache by dropping the positions that its queries
// attended to least.  Every KV head chooses for itself: the cache holds each
// head's rows apart, so position i of a compacted sequence may come from
// another token in each head, and only the number of rows has to agree.

#include <math_constants.h>

#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;

// ---- choice ----------------------------------------------------------------

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelPerSm = 4;    // CTAs per SM the register budget is sized for
constexpr int kSelBins = 2048;
constexpr int kSelCoarse = 64;  // bins per coarse count: two per lane of one warp
constexpr int kSelMaxCluster = 16;
// Keys a CTA holds in shared memory; a longer share of a row is read again
// from global memory in every pass.
constexpr int kSelMaxKeys = 48 * 1024;

// Order-preserving key of a weight: larger weight, larger key; -0 as +0; NaN
// below everything.
__device__ __forceinline__ uint32_t weight_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t k = u ^ (uint32_t)((int32_t)u >> 31 | 0x80000000);
  return x != x ? 0u : k;
}

// Steps for single lanes without a branch around each, which would keep several
// of them from being in flight.
__device__ __forceinline__ void count_if(bool go, uint32_t* bin) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared.add.u32 [%1], 1;\n\t}" ::"r"(
          (uint32_t)go),
      "r"(smem_addr(bin))
      : "memory");
}
__device__ __forceinline__ void store_if(uint32_t go, int32_t* to, int32_t x) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.b32 [%1], %2;\n\t}" ::"r"(go),
      "l"(to), "r"(x)
      : "memory");
}

// Inclusive prefix sum over a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// A cluster of CTAs per (sequence, KV head), each with an equal share of the
// row's candidates [sinks, n - recent), in order.
//
// The r-th largest key is found by radix selection in three passes (11, 11 and
// 10 bits, from the top).  Each CTA counts the digits of its keys in shared
// memory and sums them by 64; one warp per CTA adds up the cluster's 32 coarse
// counts, then the 64 bins of the coarse one that holds the wanted rank (all
// CTAs find the same digit; the coarse counts are written into every CTA's shared
// memory before the barrier, the 64 bins read from the others after it).  The keys
// stay in shared memory, so the row is read from HBM once.  Then each warp marks
// the kept keys of its contiguous part, one bit mask per 32 keys, and after a
// prefix sum over warps and CTAs writes their positions: ascending, and of the
// keys that equal the threshold the lowest positions.
//
// Bound by the chain of phases within a CTA.  With many rows (512 rows of 6-8k,
// 3.4 CTAs per SM: 14.0 us) an SM issues in 54 % of its cycles and uses 23 % of
// its shared-memory wavefronts, a fifth of them the additions (of which 39 %
// are lanes that met on a bank); of 11.1 cycles between a warp's instructions it
// waits 3.1 for weights from HBM, 1.7 for fixed latencies, 1.4 at barriers and
// 1.0 for shared memory.  With few rows (8 of 131,072 on 16 CTAs each: 13.8 us)
// the exchanges between the CTAs come on top (14.5 us with every count read from
// the others after a barrier, of which the three exchanges took 5.2).  A branch per key or
// group in place of the predicated steps cost 1.4 and 2.7 us.  No better: more
// loads in flight (15.1 against 15.5 us with 8 and 16.2 with 16, before the
// predicated steps), marking the keys that have the prefix first (14.0 and 14.4),
// 512 or 1,024 threads per CTA for few rows (15.3 and 23.6: they keep the next
// launch off the SM).
template <bool kCached>
__global__ void __launch_bounds__(kSelThreads, kSelPerSm)
    kv_evict_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[2 * kSelBins];
  // Coarse counts of every CTA of the cluster (passes alternate, as in hist), and
  // how many keys above and at the threshold each holds: written by their owners.
  __shared__ uint32_t coarse[2][kSelMaxCluster][kSelBins / kSelCoarse];
  __shared__ uint2 kept_in[kSelMaxCluster];
  __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t s_digit, s_need, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 2 * kSelBins / 4; i += kSelThreads)
    reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  grid_dep_wait();
  grid_dep_launch_dependents();
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = p.cluster, rank = C > 1 ? (int)cluster.block_rank() : 0;
  const int h = blockIdx.x / C, s = blockIdx.y;
  int n = p.context_lens[s];
  if (n < 0 || n > p.max_context_len) {
    if (tid == 0 && h == 0 && rank == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    n = n < 0 ? 0 : p.max_context_len;
  }
  const size_t row = (size_t)s * p.num_kv_heads + h;
  int32_t* keep = p.keep + row * p.budget;
  if (h == 0 && rank == 0 && tid == 0 && p.new_lens) p.new_lens[s] = min(n, p.budget);
  const int gtid = rank * kSelThreads + tid, gthreads = C * kSelThreads;
  if (n <= p.budget) {  // the same in every CTA of the cluster
    for (int i = gtid; i < p.budget; i += gthreads) keep[i] = i < n ? i : -1;
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;
  const uint32_t r = p.budget - p.sinks - p.recent;
  for (int i = gtid; i < lo; i += gthreads) keep[i] = i;
  for (int i = gtid; i < p.recent; i += gthreads) keep[p.budget - p.recent + i] = hi + i;
  if (r == 0) return;

  // This CTA's share [c0, c0 + m) of the candidates.
  const int share = ((hi - lo + C - 1) / C + 31) / 32 * 32;
  const int c0 = lo + min(rank * share, hi - lo);
  const int m = min(share, hi - c0);
  const float* w = p.weights + row * p.weights_stride + c0;
  if (C > 1) cluster.barrier_arrive();  // this CTA runs: the others may write to it
  __syncthreads();                      // the cleared histograms

  // The need-th largest among the keys that share the prefix.  Once exactly
  // that many do, all of them are kept: every key from the prefix on.
  uint32_t prefix = 0, need = r;
  bool whole = false;
#pragma unroll 1
  for (int pass = 0; pass < 3 && !whole; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t span = pass == 0 ? 0xffffffffu : (pass == 1 ? 0x1fffffu : 0x3ffu);
    uint32_t* hb = hist + (pass & 1) * kSelBins;
    // The digit of a key that has the prefix: k ^ prefix has zeros above it.
    auto count = [&](uint32_t k) {
      const uint32_t d = k ^ prefix;
      count_if(d <= span, hb + (d <= span ? d >> shift : 0u));
    };
    if (pass == 0 || !kCached) {
      // Four loads per thread are issued before any is used.
      int i0 = 0;
      for (; i0 + 4 * kSelThreads <= m; i0 += 4 * kSelThreads) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = w[i0 + j * kSelThreads + tid];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t k = weight_key(x[j]);
          if (kCached) keys[i0 + j * kSelThreads + tid] = k;
          count(k);
        }
      }
      for (int i = i0 + tid; i < m; i += kSelThreads) {
        const uint32_t k = weight_key(w[i]);
        if (kCached) keys[i] = k;
        count(k);
      }
    } else {
      const int m4 = m & ~3;
#pragma unroll 1
      for (int i = 4 * tid; i < m4; i += 8 * kSelThreads) {
        const uint4 a = *reinterpret_cast<const uint4*>(keys + i);
        // (a key that differs from the prefix above the digit is not counted)
        uint4 b = make_uint4(~prefix, ~prefix, ~prefix, ~prefix);
        if (i + 4 * kSelThreads < m4)
          b = *reinterpret_cast<const uint4*>(keys + i + 4 * kSelThreads);
        count(a.x);
        count(a.y);
        count(a.z);
        count(a.w);
        count(b.x);
        count(b.y);
        count(b.z);
        count(b.w);
      }
      if (tid < m - m4) count(keys[m4 + tid]);
    }
    __syncthreads();
    // coarse counts: 16 threads with 4 bins each
    for (int i = tid; i < kSelBins / 4; i += kSelThreads) {
      const uint4 b = reinterpret_cast<const uint4*>(hb)[i];
      uint32_t sum = (b.x + b.y) + (b.z + b.w);
#pragma unroll
      for (int d = 1; d < kSelCoarse / 4; d <<= 1) sum += __shfl_xor_sync(kFull, sum, d);
      if (i % (kSelCoarse / 4) == 0) coarse[pass & 1][rank][i / (kSelCoarse / 4)] = sum;
    }
    __syncthreads();
    if (C > 1) {
      if (pass == 0) cluster.barrier_wait();
      uint32_t* mine = &coarse[pass & 1][rank][lane];
      for (int q = warp; q < C; q += kSelWarps)
        if (q != rank) *cluster.map_shared_rank(mine, q) = *mine;
      cluster.sync();
    }
    if (warp == 0) {
      // Lane l holds coarse count 31 - l, then bins 2 (31 - l) + 1 and
      // 2 (31 - l) of the one found: prefix sums run from the largest digit.
      uint32_t c = 0;
#pragma unroll
      for (int q = 0; q < kSelMaxCluster; ++q)
        if (q < C) c += coarse[pass & 1][q][31 - lane];
      uint32_t incl = warp_scan(c);
      const int hit = __ffs(__ballot_sync(kFull, incl >= need)) - 1;
      const uint32_t rest = need - __shfl_sync(kFull, incl - c, hit);  // wanted within the 64 bins
      const int bin = (31 - hit) * kSelCoarse + 2 * (31 - lane);
      uint32_t b1 = hb[bin + 1], b0 = hb[bin];
      if (C > 1) {
        // (All loads in flight together: one after another they took 0.8 us.)
        uint2 x[kSelMaxCluster];
#pragma unroll
        for (int q = 0; q < kSelMaxCluster; ++q)
          x[q] = q < C && q != rank
                     ? *reinterpret_cast<const uint2*>(cluster.map_shared_rank(hb, q) + bin)
                     : make_uint2(0, 0);
#pragma unroll
        for (int q = 0; q < kSelMaxCluster; ++q) {
          b0 += x[q].x;
          b1 += x[q].y;
        }
      }
      incl = warp_scan(b1 + b0);
      const uint32_t before = incl - b1 - b0;
      if (before < rest && rest <= incl) {
        const bool upper = rest <= before + b1;
        s_digit = upper ? bin + 1 : bin;
        s_need = upper ? rest - before : rest - before - b1;
        s_count = upper ? b1 : b0;
      }
    }
    // The first pass's histogram is counted in again by the third: every CTA
    // is done reading it, having arrived at the second pass's barrier.
    if (pass == 1)
      for (int i = tid; i < kSelBins / 4; i += kSelThreads)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    prefix |= s_digit << shift;
    need = s_need;
    whole = s_count == need;
  }

  // Each warp marks the kept keys of a contiguous part of the share, in whole
  // 32-key groups, 32 groups at a time: lane g holds the mask of group g.
  const int part = ((m + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(warp * part, m), w1 = min(w0 + part, m);
  auto masks = [&](int base, uint32_t least) {  // of keys of at least this value
    uint32_t mine = 0;
    const int groups = min(32, (w1 - base + 31) / 32);
    for (int g = 0; g < groups; g += 8) {
      uint32_t k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = base + 32 * (g + j) + lane;
        k[j] = i >= w1 ? 0u : (kCached ? keys[i] : weight_key(w[i]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = __ballot_sync(kFull, k[j] >= least);
        if (lane == g + j) mine = a;
      }
    }
    // (a key past the part's end reads as 0, which `least` may be)
    const int left = w1 - base - 32 * lane;
    return left >= 32 ? mine : (left > 0 ? mine & ((1u << left) - 1u) : 0u);
  };
  // Two thresholds only where some, but not all, of the keys that equal the
  // prefix are kept (then it is a whole key; NaN's 0 has none below it).
  uint32_t gt = 0, eq = 0;
  auto count_kept = [&](int base, uint32_t& gm, uint32_t& em) {
    const uint32_t ge = masks(base, prefix);
    gm = whole ? ge : (prefix == 0xffffffffu ? 0u : masks(base, prefix + 1));
    em = ge & ~gm;
  };
  uint32_t gm = 0, em = 0;
  for (int base = w0; base < w1; base += 1024) {
    count_kept(base, gm, em);
    gt += __popc(gm);
    eq += __popc(em);
  }
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  const uint32_t sg = warp_scan(lane < kSelWarps ? warp_gt[lane] : 0u);
  const uint32_t se = warp_scan(lane < kSelWarps ? warp_eq[lane] : 0u);
  uint32_t above = warp > 0 ? __shfl_sync(kFull, sg, warp - 1) : 0u;
  uint32_t equal = warp > 0 ? __shfl_sync(kFull, se, warp - 1) : 0u;
  if (C > 1) {
    const uint32_t tg = __shfl_sync(kFull, sg, 31), te = __shfl_sync(kFull, se, 31);
    if (warp == 0 && lane < C) *cluster.map_shared_rank(&kept_in[rank], lane) = make_uint2(tg, te);
    cluster.sync();  // (no CTA reads another's memory from here on)
    const uint2 x = lane < rank ? kept_in[lane] : make_uint2(0, 0);
    above += __reduce_add_sync(kFull, x.x);
    equal += __reduce_add_sync(kFull, x.y);
  }
  const uint32_t below = (1u << lane) - 1u;
  int32_t* to = keep + lo;
  uint32_t at = above + min(equal, need);  // kept so far
  for (int base = w0; base < w1; base += 1024) {
    if (part > 1024) count_kept(base, gm, em);
    if (!whole) {
      // The group's ties before the need-th: the lowest bits of its mask.
      const uint32_t ties = __popc(em);
      const uint32_t eb = equal + warp_scan(ties) - ties;
      uint32_t take = eb < need ? em : 0u;
      for (uint32_t extra = eb < need ? max(ties, need - eb) - (need - eb) : 0u; extra > 0; --extra)
        take &= ~(0x80000000u >> __clz(take));
      gm |= take;
      equal += __reduce_add_sync(kFull, ties);
    }
    const uint32_t kept = __popc(gm);
    const uint32_t incl = warp_scan(kept);
    const uint32_t first = at + incl - kept;
    const int groups = min(32, (w1 - base + 31) / 32);
    for (int g = 0; g < groups; g += 8) {  // (the mask of a group past the last is 0)
      uint32_t k[8], f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[j] = __shfl_sync(kFull, gm, g + j);
        f[j] = __shfl_sync(kFull, first, g + j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        store_if(k[j] >> lane & 1u, to + f[j] + __popc(k[j] & below),
                 c0 + base + 32 * (g + j) + lane);
    }
    at += __shfl_sync(kFull, incl, 31);
  }
}

// ---- compaction ------------------------------------------------------------

// A CTA of one to eight warps moves K or V of one (sequence, KV head), or its
// weights, from the front, 32 rows (a tile) per warp and round, through a ring of
// tiles in shared memory for each warp:
// rows are gathered by 16-byte asynchronous copies, and the kept rows of a
// destination block, which lie side by side, go out as one bulk copy.
//
// keep[i] ascends and is at least i.  With rows moved in place a tile's sources
// then lie at or behind its destinations and the next tiles' sources behind them
// all: a round may be stored as soon as its own loads have landed, whatever loads
// of later rounds are in flight.
//
// Bound by HBM.  64 sequences x 8 heads, 6-8k positions of 128 cut to 2k (1.1 GB
// in all): 217 us (75 % of the copy rate) with tiles in registers and a barrier
// between a tile's loads and its stores, whatever the rows or bytes in flight;
// 326 us with a bulk copy per row, in and out (an SM starts one about every 23
// cycles); 180 us so (91 %).  With few pairs a CTA's chain of rounds bounds it:
// one sequence x 8 heads cut from 131,072 to 32,768 takes 195 us on eight warps
// per CTA (1.4 TB/s), 466 us on one.
constexpr int kCmpMaxWarps = 8;
constexpr int kCmpMinStages = 3, kCmpMaxStages = 8;
constexpr int kCmpSmBytes = 226 * 1024;   // shared memory of an SM
constexpr int kCmpFixedBytes = 1024 + kCmpMaxWarps * kCmpMaxStages * 8;  // of a CTA beside its rings

__device__ __forceinline__ void bulk_store(void* dst, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_addr(src_smem)), "r"(bytes)
               : "memory");
}

// The weights, 16 per thread and step: the kept positions are read two steps
// ahead and the values one step ahead of the step that is stored (which, as with
// rows, only its own loads have to precede).
__device__ __forceinline__ void compact_weights(const CompactParams& p, const int32_t* keep,
                                                float* w, int n, int m) {
  constexpr int kPer = 16;
  const int threads = blockDim.x, step = threads * kPer, tid = threadIdx.x;
  int k[kPer];
  bool here[kPer], next[kPer];
  float x[kPer], y[kPer];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + u * threads + tid;
      k[u] = i < m ? __ldg(keep + i) : -1;
    }
  };
  auto read = [&](int i0) {  // the values of the positions in k
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + u * threads + tid;
      next[u] = k[u] >= i && k[u] < n;  // (never where there is no entry: k is -1)
      if (i < m && !next[u]) atomicOr(p.status, PKV_DEV_BAD_KEEP);
      y[u] = next[u] ? __ldcg(w + k[u]) : 0.f;
    }
  };
  fetch(0);
  read(0);
  fetch(step);
  for (int i0 = 0; i0 < m; i0 += step) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      x[u] = y[u];
      here[u] = next[u];
    }
    if (i0 + step < m) {
      read(i0 + step);
      fetch(i0 + 2 * step);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (here[u]) w[i0 + u * threads + tid] = x[u];
  }
  __syncthreads();
#pragma unroll 8
  for (int i = m + tid; i < n; i += threads) w[i] = 0.f;
}

template <int CPR>  // 16-byte chunks per row
__global__ void __launch_bounds__(kCmpMaxWarps * 32) kv_compact_kernel(const CompactParams p,
                                                                      int stages) {
  constexpr int kRowBytes = CPR * 16;
  constexpr int kStageBytes = 32 * kRowBytes + 32 * 8;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[kCmpMaxWarps * kCmpMaxStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // This warp's ring: [stages][32] rows, and where each row goes (nullptr: it
  // does not move).
  unsigned char* ring = smem + warp * stages * kStageBytes;
  unsigned char*(*to_ring)[32] =
      reinterpret_cast<unsigned char*(*)[32]>(ring + stages * 32 * kRowBytes);
  uint64_t* full = bars + warp * stages;
  if (lane == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 32);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int h = blockIdx.x, s = blockIdx.y, job = blockIdx.z;  // 0: K, 1: V, 2: weights
  int n = p.context_lens[s];
  if (n < 0 || n > p.max_len) {
    if (threadIdx.x == 0 && h == 0 && job == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    n = n < 0 ? 0 : p.max_len;
  }
  const int m = min(n, p.budget);
  const size_t row = (size_t)s * p.num_kv_heads + h;
  const int32_t* keep = p.keep + row * p.budget;
  if (job == 2) {
    compact_weights(p, keep, p.weights + row * p.weights_stride, n, m);
    return;
  }

  unsigned char* cache = static_cast<unsigned char*>(job == 1 ? p.v_cache : p.k_cache);
  const int32_t* src_row = p.src_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* dst_row = p.dst_tables + (size_t)s * p.dst_blocks_per_seq;
  const int mask = p.block_size - 1;
  // The warp's q-th tile is tile q * warps + warp; a round is one tile per warp.
  const int rounds = ((m + 31) / 32 + warps - 1) / warps;
  auto first_row = [&](int q) { return (q * warps + warp) * 32; };
  auto at = [&](int block, int pos) {
    return cache +
           (((long long)block * p.num_kv_heads + h) * p.block_size + (pos & mask)) * kRowBytes;
  };
  // The lane's rows of the next tiles to load, four tiles (a group) at a time:
  // kept positions and destination blocks are read two groups ahead, source
  // blocks (which depend on the positions) one group ahead.
  struct Group {
    int k[4], sb[4], db[4];  // k < 0: no row
  } cur, nxt, fut;
  auto fetch = [&](int g) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = first_row(g * 4 + u) + lane;
      fut.k[u] = i < m ? __ldg(keep + i) : -1;
      fut.db[u] = i < m ? __ldg(dst_row + (i >> p.log2_block)) : 0;
    }
  };
  auto resolve = [&](int g) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = first_row(g * 4 + u) + lane;
      const bool good = fut.k[u] >= i && fut.k[u] < n;
      if (i < m && !good) atomicOr(p.status, PKV_DEV_BAD_KEEP);
      nxt.k[u] = i < m && good ? fut.k[u] : -1;
      nxt.db[u] = fut.db[u];
      nxt.sb[u] = nxt.k[u] >= 0 ? __ldg(src_row + (fut.k[u] >> p.log2_block)) : 0;
    }
  };
  fetch(0);
  resolve(0);
  fetch(1);
  auto load = [&](int q, int st) {
    const int i = first_row(q) + lane, u = q & 3;
    if (u == 0) {
      cur = nxt;
      resolve(q / 4 + 1);
      fetch(q / 4 + 2);
    }
    int k = cur.k[0], sb = cur.sb[0], db = cur.db[0];
#pragma unroll
    for (int v = 1; v < 4; ++v)
      if (u == v) {
        k = cur.k[v];
        sb = cur.sb[v];
        db = cur.db[v];
      }
    bool moves = k >= 0;
    if (moves &&
        ((unsigned)sb >= (unsigned)p.num_blocks || (unsigned)db >= (unsigned)p.num_blocks)) {
      atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
      moves = false;
    }
    moves = moves && (sb != db || k != i);
    to_ring[st][lane] = moves ? at(db, i) : nullptr;
    const unsigned who = __ballot_sync(kFull, moves);
    const unsigned long long from =
        reinterpret_cast<unsigned long long>(moves ? at(sb, k) : cache);
    // 32 / CPR rows per step: CPR lanes with one chunk each.
    const uint32_t to = smem_addr(ring) + (uint32_t)(st * 32 * kRowBytes) + lane * 16;
#pragma unroll
    for (int c = 0; c < CPR; ++c) {
      const int r = c * (32 / CPR) + lane / CPR;
      const unsigned long long src = __shfl_sync(kFull, from, r) + lane % CPR * 16;
      if (who >> r & 1u)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + c * 512), "l"(src)
                     : "memory");
    }
    // Every lane arrives once its copies have landed.
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                     smem_addr(&full[st]))
                 : "memory");
  };
  int ahead = 0, ahead_st = 0;  // the next tile to load and its stage
  auto load_next = [&]() {
    load(ahead++, ahead_st);
    if (++ahead_st == stages) ahead_st = 0;
  };
  while (ahead < min(stages - 2, rounds)) load_next();
  const int seg = min(p.block_size, 32);  // rows of a tile in one destination block
  const unsigned seg_bits = (seg == 32 ? kFull : (1u << seg) - 1u) << (lane & ~(seg - 1));
  int st = 0, phase = 0;
  bool ok = true;
  for (int q = 0; q < rounds; ++q) {
    if (ok && ahead < rounds) {
      // Its stage was last read by the stores of tile q - 2, of which this lane's
      // are done once at most its newest group is not.
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
      load_next();
    }
    // (A wait that gives up, never expected, leaves ok false: the loop runs on
    // without copies, so that the barriers stay matched.)
    if (ok && !mbar_wait_warp(&full[st], phase, p.status)) ok = false;
    if (warps > 1) __syncthreads();  // every warp's tile of the round has landed
    if (ok) {
      // The rows were written by plain copies: order them before the bulk copy.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      unsigned char* to = to_ring[st][lane];
      const unsigned who = __ballot_sync(kFull, to != nullptr);
      const int left = m - first_row(q);
      const unsigned there = left >= 32 ? kFull : (left > 0 ? (1u << left) - 1u : 0u);
      const unsigned char* src = ring + (st * 32 + lane) * kRowBytes;
      if ((who & seg_bits) == (there & seg_bits)) {  // the block's rows side by side
        if (to && (lane & (seg - 1)) == 0) bulk_store(to, src, __popc(who & seg_bits) * kRowBytes);
      } else if (to) {
        bulk_store(to, src, kRowBytes);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
  // Copies still in flight at exit land first (loads: only after a timeout).
  if (!ok) asm volatile("cp.async.wait_all;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

namespace {

// A launch of kv_evict_select_kernel as clusters of `cluster` CTAs.
struct SelectLaunch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  SelectLaunch(int rows_x, int rows_y, int cluster, size_t smem, cudaStream_t stream) : cfg{} {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(rows_x * cluster, rows_y);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// The largest cluster that the device (or the part of it this process may use)
// places with the most shared memory a CTA asks for.
int largest_cluster(cudaStream_t stream) {
  for (int c = kSelMaxCluster; c > 1; c /= 2) {
    SelectLaunch l(1, 1, c, (size_t)kSelMaxKeys * 4, stream);
    int fit = 0;
    const cudaError_t err =
        cudaOccupancyMaxActiveClusters(&fit, kv_evict_select_kernel<true>, &l.cfg);
    if (err != cudaSuccess) (void)cudaGetLastError();
    if (err == cudaSuccess && fit > 0) return c;
  }
  return 1;
}

}  // namespace

cudaError_t launch_kv_evict_select(SelectParams p, int num_seqs, int sm_count,
                                   cudaStream_t stream) {
  static int largest[64] = {};  // largest_cluster of a device; 0: not asked yet
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  int most = dev < 64 ? __atomic_load_n(&largest[dev], __ATOMIC_ACQUIRE) : 0;
  if (most == 0) {
    err = cudaFuncSetAttribute(kv_evict_select_kernel<true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxKeys * 4);
    for (auto k : {kv_evict_select_kernel<true>, kv_evict_select_kernel<false>})
      if (err == cudaSuccess)
        err = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    most = largest_cluster(stream);
    if (dev < 64) __atomic_store_n(&largest[dev], most, __ATOMIC_RELEASE);
  }
  // CTAs per row: as many as keep the whole launch within one wave, each with
  // 1,024 keys or more.  (8 rows of 131,072: 95 us on one CTA each with 1,024
  // threads, 33 us on 8, 14 us on 16.)
  const long long rows = (long long)num_seqs * p.num_kv_heads;
  int cluster = 1;
  while (cluster < most && rows * cluster * 2 <= (long long)kSelPerSm * sm_count &&
         p.max_context_len / (cluster * 2) >= 1024)
    cluster *= 2;
  p.cluster = cluster;
  const int share = (std::max(1, (p.max_context_len + cluster - 1) / cluster) + 31) / 32 * 32;
  const bool cached = share <= kSelMaxKeys;
  auto kernel = cached ? kv_evict_select_kernel<true> : kv_evict_select_kernel<false>;
  SelectLaunch l(p.num_kv_heads, num_seqs, cluster, cached ? (size_t)share * 4 : 0, stream);
  err = cudaLaunchKernelEx(&l.cfg, kernel, p);
  const cudaError_t last = cudaGetLastError();  // clears the error, as after <<<>>>
  return err != cudaSuccess ? err : last;
}

cudaError_t launch_kv_compact(const CompactParams& p, int num_seqs, int sm_count,
                              cudaStream_t stream) {
  // One warp alone moves about 40 GB/s: as many warps per CTA as give the launch
  // seven per SM (which filled HBM), and for each a ring of as many tiles as the
  // SM's shared memory holds for its share of the CTAs, so that all run at once.
  const long long ctas = 2LL * p.num_kv_heads * num_seqs;
  int warps = 1;
  while (warps < kCmpMaxWarps && ctas * warps * 2 <= 7LL * sm_count) warps *= 2;
  const int stage = 32 * p.head_dim * 2 + 32 * 8;
  const long long per_sm = (ctas + sm_count - 1) / sm_count;
  const long long room = (kCmpSmBytes / per_sm - kCmpFixedBytes) / warps;
  const int stages = (int)std::max<long long>(
      kCmpMinStages, std::min<long long>(kCmpMaxStages, room / stage));
  const dim3 grid(p.num_kv_heads, num_seqs, p.weights ? 3 : 2);
  auto kernel = p.head_dim == 64 ? kv_compact_kernel<8> : kv_compact_kernel<16>;
  static unsigned long long configured = 0;  // bit per device ordinal (< 64)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    for (auto k : {kv_compact_kernel<8>, kv_compact_kernel<16>}) {
      err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kCmpSmBytes - kCmpFixedBytes);
      if (err != cudaSuccess) return err;
    }
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  return launch_overlapped(kernel, grid, dim3(32 * warps), (size_t)warps * stages * stage, stream,
                           p, stages);
}

}  // namespace pkv
