// Eviction from the paged cache: which positions a sequence keeps
// (kv_evict_select) and the move of their rows to the front (kv_compact).
//
// A sequence keeps a bounded cache by dropping the positions that its queries
// attended to least.  Every KV head chooses for itself: the cache holds each
// head's rows apart, so position i of a compacted sequence may come from
// another token in each head, and only the number of rows has to agree.

#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ---- choice ----------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 4;  // elements per thread and tile of the output pass

// Order-preserving key of a weight: larger weight, larger key; -0 as +0; NaN
// below everything.
__device__ __forceinline__ uint32_t weight_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the CTA's threads; *total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t w = warp_sums[lane];  // 32 warps
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, w, d);
    if (lane >= d) w += y;
  }
  const uint32_t before = warp > 0 ? __shfl_sync(kFull, w, warp - 1) : 0u;
  *total = __shfl_sync(kFull, w, 31);
  __syncthreads();
  return before + x - v;
}

// One CTA per (sequence, KV head).  The r-th largest of the m candidates is
// found by a radix selection over the keys, 8 bits a pass, and the kept
// positions are written in ascending order by a prefix sum.
__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const SelectParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_digit, s_need;
  const int h = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x;
  int n = p.context_lens[s];
  if (n < 0 || n > p.max_context_len) {
    if (tid == 0 && h == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    n = n < 0 ? 0 : p.max_context_len;
  }
  const size_t row = (size_t)s * p.num_kv_heads + h;
  int32_t* keep = p.keep + row * p.budget;
  if (h == 0 && tid == 0 && p.new_lens) p.new_lens[s] = min(n, p.budget);
  if (n <= p.budget) {
    for (int i = tid; i < p.budget; i += kSelThreads) keep[i] = i < n ? i : -1;
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;
  const uint32_t r = p.budget - p.sinks - p.recent;
  for (int i = tid; i < lo; i += kSelThreads) keep[i] = i;
  for (int i = tid; i < p.recent; i += kSelThreads) keep[p.budget - p.recent + i] = hi + i;
  if (r == 0) return;
  const float* w = p.weights + row * p.weights_stride;

  uint32_t prefix = 0, need = r;  // the need-th largest among keys that share the prefix
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    // thread d holds bin 255 - d: the prefix sum runs from the largest keys
    const uint32_t c = tid < 256 ? hist[255 - tid] : 0u;
    uint32_t total;
    const uint32_t before = block_scan(c, warp_sums, &total);
    if (tid < 256 && before < need && need <= before + c) {
      s_digit = 255 - tid;
      s_need = need - before;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    need = s_need;
    __syncthreads();
  }
  // Kept: every key above prefix, and the first `need` that equal it.
  uint32_t out = lo, ties = 0;
  for (int i0 = lo; i0 < hi; i0 += kSelThreads * kSelPer) {
    uint32_t k[kSelPer];
    uint32_t mine = 0;  // keys above in the low half, equal ones in the high half
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) {
      const int i = i0 + tid * kSelPer + j;
      k[j] = i < hi ? weight_key(w[i]) : 0u;
      if (i < hi) mine += k[j] > prefix ? 1u : (k[j] == prefix ? 65536u : 0u);
    }
    uint32_t total;
    const uint32_t before = block_scan(mine, warp_sums, &total);
    uint32_t above = before & 0xffffu, equal = ties + (before >> 16);
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) {
      const int i = i0 + tid * kSelPer + j;
      if (i >= hi) break;
      const bool eq = k[j] == prefix;
      if (k[j] > prefix || (eq && equal < need)) {
        // ties placed before this tile are part of `out` already
        const uint32_t placed = min(equal, need) - min(ties, need);
        keep[out + above + placed] = i;
      }
      above += k[j] > prefix;
      equal += eq;
    }
    const uint32_t tile_ties = total >> 16;
    out += (total & 0xffffu) + min(ties + tile_ties, need) - min(ties, need);
    ties += tile_ties;
  }
}

// ---- compaction ------------------------------------------------------------

constexpr int kCmpThreads = 256;
constexpr int kCmpChunks = 4;                  // 16-byte chunks of a row per CTA: a 64-byte slice
constexpr int kCmpRows = kCmpThreads / kCmpChunks;
constexpr int kCmpUnroll = 4;                  // rows in flight per thread

// A CTA moves one 64-byte column slice of K or of V of one (sequence, KV
// head), or its weights, tile by tile from the front.  keep[i] ascends and is
// at least i, so with rows moved in place a tile's sources lie at or behind
// its destinations and the next tile's sources behind them all: one barrier
// between a tile's loads and its stores is enough.
__global__ void __launch_bounds__(kCmpThreads) kv_compact_kernel(const CompactParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int tid = threadIdx.x;
  const int h = blockIdx.y, s = blockIdx.z;
  int n = p.context_lens[s];
  if (n < 0 || n > p.max_len) {
    if (tid == 0 && h == 0 && blockIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    n = n < 0 ? 0 : p.max_len;
  }
  const int m = min(n, p.budget);
  const size_t row = (size_t)s * p.num_kv_heads + h;
  const int32_t* keep = p.keep + row * p.budget;
  const int slices = p.head_dim * 2 / 16 / kCmpChunks;  // of one row

  if ((int)blockIdx.x >= 2 * slices) {  // the weights
    float* w = p.weights + row * p.weights_stride;
    for (int i0 = 0; i0 < m; i0 += kCmpThreads * kCmpUnroll) {
      float x[kCmpUnroll];
      bool ok[kCmpUnroll];
#pragma unroll
      for (int u = 0; u < kCmpUnroll; ++u) {
        const int i = i0 + u * kCmpThreads + tid;
        const int k = i < m ? keep[i] : -1;
        ok[u] = i < m && k >= i && k < n;
        if (i < m && !ok[u]) atomicOr(p.status, PKV_DEV_BAD_KEEP);
        x[u] = ok[u] ? w[k] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kCmpUnroll; ++u)
        if (ok[u]) w[i0 + u * kCmpThreads + tid] = x[u];
    }
    __syncthreads();
    for (int i = m + tid; i < n; i += kCmpThreads) w[i] = 0.f;
    return;
  }

  const bool is_v = (int)blockIdx.x >= slices;
  uint4* cache = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache);
  const int cpr = p.head_dim * 2 / 16;
  const int c = ((int)blockIdx.x - (is_v ? slices : 0)) * kCmpChunks + tid % kCmpChunks;
  const int32_t* src_row = p.src_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* dst_row = p.dst_tables + (size_t)s * p.dst_blocks_per_seq;
  const int lane_row = tid / kCmpChunks;
  const int mask = p.block_size - 1;
  for (int i0 = 0; i0 < m; i0 += kCmpRows * kCmpUnroll) {
    uint4 x[kCmpUnroll];
    long long to[kCmpUnroll];
#pragma unroll
    for (int u = 0; u < kCmpUnroll; ++u) {
      const int i = i0 + u * kCmpRows + lane_row;
      to[u] = -1;
      if (i >= m) continue;
      const int k = keep[i];
      if (k < i || k >= n) {
        atomicOr(p.status, PKV_DEV_BAD_KEEP);
        continue;
      }
      const int sb = src_row[k >> p.log2_block], db = dst_row[i >> p.log2_block];
      if ((unsigned)sb >= (unsigned)p.num_blocks || (unsigned)db >= (unsigned)p.num_blocks) {
        atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
        continue;
      }
      if (sb == db && k == i) continue;  // already in place
      x[u] = cache[(((long long)sb * p.num_kv_heads + h) * p.block_size + (k & mask)) * cpr + c];
      to[u] = (((long long)db * p.num_kv_heads + h) * p.block_size + (i & mask)) * cpr + c;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCmpUnroll; ++u)
      if (to[u] >= 0) cache[to[u]] = x[u];
  }
}

}  // namespace

cudaError_t launch_kv_evict_select(const SelectParams& p, int num_seqs, cudaStream_t stream) {
  return launch_overlapped(kv_evict_select_kernel, dim3(p.num_kv_heads, num_seqs),
                           dim3(kSelThreads), 0, stream, p);
}

cudaError_t launch_kv_compact(const CompactParams& p, int num_seqs, cudaStream_t stream) {
  const int slices = 2 * (p.head_dim * 2 / 16 / kCmpChunks) + (p.weights ? 1 : 0);
  return launch_overlapped(kv_compact_kernel, dim3(slices, p.num_kv_heads, num_seqs),
                           dim3(kCmpThreads), 0, stream, p);
}

}  // namespace pkv
