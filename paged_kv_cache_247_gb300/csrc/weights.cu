// Accumulated attention weights: how much weight each cached position has
// received from the queries, per KV head, summed over the query heads of its
// group.  Both kernels here run after the attention itself and use what it
// left behind: the base-2 logits and softmax statistics of a decode step, the
// log-sum of each query row of a prompt chunk.
//
//   weights[s][h][t] = decay * weights[s][h][t] + sum_rows 2^(x_row(t) - lse_row)
//
// with x the logit in base 2 and lse = m + log2(l) the row's log-sum.

#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace tc;

// decay 0 drops what was there, whatever it was (it may never have been set).
__device__ __forceinline__ float decayed(float decay, float old, float add) {
  return decay == 0.f ? add : fmaf(decay, old, add);
}

// ---- decode ----------------------------------------------------------------

constexpr int kDwThreads = 256;
constexpr int kDwPer = 4;  // positions per thread
constexpr int kDwSpan = kDwThreads * kDwPer;

// One CTA per (1024 positions, KV head, sequence).  The partitions' (m, l) of
// each query head of the group give its log-sum; the logits are read once.
__global__ void __launch_bounds__(kDwThreads) decode_weights_kernel(const DecodeParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float lse[kMaxTcGroup];
  const int s = blockIdx.z, kvh = blockIdx.y;
  const int t0 = blockIdx.x * kDwSpan;
  const long long cap = min((long long)p.max_context_len,
                            (long long)p.max_blocks_per_seq * p.block_size);
  int ctx = p.context_lens[s];
  ctx = ctx < 0 ? 0 : (ctx > cap ? (int)cap : ctx);
  if (t0 >= ctx) return;
  const int np = (ctx + p.partition_size - 1) / p.partition_size;
  const size_t row0 = (size_t)s * p.num_q_heads + (size_t)kvh * p.group;
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < p.group; g += kDwThreads / 32) {
    const float* mr = p.ws_m + (row0 + g) * p.num_parts;
    const float* lr = p.ws_l + (row0 + g) * p.num_parts;
    float M = -CUDART_INF_F;
    for (int i = lane; i < np; i += 32) M = fmaxf(M, mr[i]);
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, mk));
    float l = 0.f;
    for (int i = lane; i < np; i += 32) l += lr[i] * exp2f(mr[i] - M);
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) l += __shfl_xor_sync(0xffffffffu, l, mk);
    if (lane == 0) lse[g] = M + log2f(l);
  }
  __syncthreads();
  float sum[kDwPer];
#pragma unroll
  for (int j = 0; j < kDwPer; ++j) sum[j] = 0.f;
  const float* x = p.ws_x + row0 * p.x_stride + t0;
#pragma unroll 4
  for (int g = 0; g < p.group; ++g) {
#pragma unroll
    for (int j = 0; j < kDwPer; ++j) {
      const int t = j * kDwThreads + threadIdx.x;
      if (t0 + t < ctx) sum[j] += exp2f(x[(size_t)g * p.x_stride + t] - lse[g]);
    }
  }
  float* w = p.weights + ((size_t)s * p.num_kv_heads + kvh) * p.weights_stride + t0;
#pragma unroll
  for (int j = 0; j < kDwPer; ++j) {
    const int t = j * kDwThreads + threadIdx.x;
    if (t0 + t < ctx) w[t] = decayed(p.decay, w[t], sum[j]);
  }
}

// ---- prompt chunks ---------------------------------------------------------
//
// One CTA per (128-key tile, KV head, sequence): S^T = K_tile . Q^T with the
// keys as the MMA's M dimension (one tensor-memory lane per key) and 128
// (query, head) rows as N, for every tile of query rows that sees the keys.
// A thread adds up its key's row of 2^(x - lse): no exchange between threads,
// no atomics, and the same order of additions whatever runs beside it.
//
//   warps 0-3  the sums, one thread per key
//   warp 4     producer: the K tile once, then the Q tiles into a ring
//   warp 5     issues the products; owns the tensor memory (two S^T buffers)

constexpr int kKeys = kTileKeys;
constexpr int kRows = 128;  // query rows per tile: MMA N
constexpr int kSumThreads = 128;
constexpr int kPwThreads = kSumThreads + 64;
constexpr int kPwTmem = 256;

template <int D>
struct PwSmem {
  static constexpr int kGroup = (D / 64) * 1024;
  static constexpr int kTile = (kKeys / 8) * kGroup;  // K tile and Q tile alike
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = kTile;
  static constexpr int kLse = kQ + kStages * kTile;  // [2][kRows] floats
  static constexpr int kPos = kLse + 2 * kRows * 4;  // [2][kRows] ints
  static constexpr int kBar = kPos + 2 * kRows * 4;
  static constexpr int kTmemSlot = kBar + 16 * 8;
  static constexpr int kBytes = kTmemSlot + 16 + 1024;  // + alignment slack
};

template <typename T, int D>
__global__ void __launch_bounds__(kPwThreads, 2)
    prefill_weights_kernel(const PrefillWeightsParams p, const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap) {
  using L = PwSmem<D>;
  constexpr int S = L::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sK = smem;
  unsigned char* sQ = smem + L::kQ;
  float* s_lse = reinterpret_cast<float*>(smem + L::kLse);
  int* s_pos = reinterpret_cast<int*>(smem + L::kPos);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = k_full + 1;   // [S] Q tile landed
  uint64_t* q_empty = q_full + S;  // [S] products done reading it (commit)
  uint64_t* s_full = q_empty + S;  // [2] S^T buffer computed (commit)
  uint64_t* s_free = s_full + 2;   // [2] S^T buffer read
  uint64_t* drain = s_free + 2;
  static_assert(2 * S + 6 <= 16, "barrier area too small");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kt = blockIdx.x % p.key_tiles;
  const int pair = blockIdx.x / p.key_tiles;
  const int kvh = pair % p.num_kv_heads, s = pair / p.num_kv_heads;
  const int G = p.group, Gp = p.group_pow2, qpt = kRows / Gp;

  const int q0 = p.query_start[s];
  const int nq = p.query_start[s + 1] - q0;
  int ctx = p.context_lens[s];
  const long long cap = min((long long)p.max_context_len,
                            (long long)p.max_blocks_per_seq * p.block_size);
  if (nq <= 0 || ctx < nq) return;  // flagged by the attention kernel
  if (ctx > cap) ctx = (int)cap;
  const int key0 = kt * kKeys;
  if (key0 >= ctx) return;
  // Queries j_lo .. nq - 1 count and see the tile (the last one always does).
  const int first = p.window > 0 ? max(0, nq - p.window) : 0;
  const int j_lo = max(first, key0 - (ctx - nq));
  const int n_tiles = (nq - j_lo + qpt - 1) / qpt;

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], kSumThreads);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kPwTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------------------- producer
    const int B = p.block_size;
    const int R = B < kKeys ? B : kKeys;
    const int nseg = (min(ctx - key0, kKeys) + R - 1) / R;
    const int key = key0 + lane * R;
    int phys = lane < nseg ? __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + key / B) : 0;
    if ((unsigned)phys >= (unsigned)p.num_blocks) phys = 0;  // flagged by the attention kernel
    if (lane == 0) mbar_arrive_expect_tx(k_full, (uint32_t)nseg * R * D * (uint32_t)sizeof(T));
    __syncwarp();
    if (lane < nseg)
      tma_load_group(sK + lane * (R / 8) * L::kGroup, &kmap,
                     ((phys * p.num_kv_heads + kvh) * B + key % B) / 8, k_full);
    int issued = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int st = i % S;
      if (i >= S && !mbar_wait_warp(&q_empty[st], ((i / S) - 1) & 1, p.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[st], L::kTile);
        tma_load_token_heads(sQ + st * L::kTile, &qmap, kvh * G, q0 + j_lo + i * qpt, &q_full[st]);
      }
      __syncwarp();
      issued = i + 1;
    }
    // Copies still in flight at exit (only after a timeout) land first.
    mbar_drain(k_full, 0);
    for (int i = issued > S ? issued - S : 0; i < issued; ++i)
      mbar_drain(&q_full[i % S], (i / S) & 1);
    __syncwarp();
  } else if (warp == 5) {
    // --------------------------------------------------------------- issuer
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t idesc = instr_desc(bf16, false, false, kRows, kKeys);
    const uint32_t aK = smem_addr(sK), aQ = smem_addr(sQ);
    bool ok = mbar_wait_warp(k_full, 0, p.status);
    for (int i = 0; ok && i < n_tiles; ++i) {
      const int st = i % S, b = i & 1;
      if (!mbar_wait_warp(&q_full[st], (i / S) & 1, p.status) ||
          (i >= 2 && !mbar_wait_warp(&s_free[b], ((i >> 1) - 1) & 1, p.status)))
        break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_f16_ss_warp(tmem + b * kRows,
                        smem_desc(aK + (ks / 4) * 1024 + (ks % 4) * 32, 16, L::kGroup),
                        smem_desc(aQ + st * L::kTile + (ks / 4) * (kRows * 128) + (ks % 4) * 32, 16,
                                  1024),
                        idesc, ks > 0 ? 1u : 0u);
      mma_commit_warp(&s_full[b]);
      mma_commit_warp(&q_empty[st]);
    }
    mma_commit_warp(drain);
    mbar_drain(drain, 0);
    __syncwarp();
  } else {
    // ----------------------------------------------------------------- sums
    const int t = threadIdx.x;
    const int key = key0 + t;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const float qs = p.qscale;
    float acc = 0.f, lost = 0.f;  // compensated: the low part of the running sum
    bool ok = true;
    for (int i = 0; i < n_tiles; ++i) {
      const int b = i & 1;
      const int j0 = j_lo + i * qpt;
      {  // column t of the tile: query row j, head g
        const int j = j0 + t / Gp, g = t % Gp;
        const bool there = j < nq && g < G && q0 + j < p.total_queries;
        s_lse[b * kRows + t] =
            there ? p.lse[(size_t)(q0 + j) * p.num_q_heads + kvh * G + g] : CUDART_INF_F;
        s_pos[b * kRows + t] = there ? ctx - nq + j : -1;
      }
      named_barrier_sync(1, kSumThreads);
      if (ok && !mbar_wait_warp(&s_full[b], (i >> 1) & 1, p.status)) ok = false;
      tc_fence_after();
      float sum = 0.f;
#pragma unroll
      for (int c0 = 0; c0 < kRows; c0 += 32) {
        float x[32];
        tmem_ld32f(tmem + b * kRows + c0 + lane_base, x);
        tmem_wait_ld_bind(x);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float e = ex2(fmaf(x[c], qs, -s_lse[b * kRows + c0 + c]));
          part[c & 3] += key <= s_pos[b * kRows + c0 + c] ? e : 0.f;
        }
        sum += (part[0] + part[1]) + (part[2] + part[3]);
      }
      tc_fence_before();
      mbar_arrive(&s_free[b]);
      const float y = sum - lost;
      const float z = acc + y;
      lost = (z - acc) - y;
      acc = z;
    }
    if (ok && key < ctx) {
      float* w = p.weights + ((size_t)s * p.num_kv_heads + kvh) * p.weights_stride + key;
      *w = decayed(p.decay, *w, acc);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kPwTmem));
  }
}

template <typename T, int D>
cudaError_t launch_pw_typed(const PrefillWeightsParams& p, const CUtensorMap& qm,
                            const CUtensorMap& km, int ctas, cudaStream_t stream) {
  using L = PwSmem<D>;
  static unsigned long long configured = 0;  // bit per device ordinal (< 64)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    err = cudaFuncSetAttribute(prefill_weights_kernel<T, D>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (err != cudaSuccess) return err;
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  prefill_weights_kernel<T, D><<<ctas, kPwThreads, L::kBytes, stream>>>(p, qm, km);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeParams& p, cudaStream_t stream) {
  const dim3 grid((p.max_context_len + kDwSpan - 1) / kDwSpan, p.num_kv_heads, p.num_seqs);
  return launch_overlapped(decode_weights_kernel, grid, dim3(kDwThreads), 0, stream, p);
}

cudaError_t launch_prefill_weights(const PrefillArgs& a, cudaStream_t stream, bool* unsupported) {
  *unsupported = false;
  PrefillWeightsParams p{};
  p.lse = a.lse;
  p.weights = a.weights;
  p.weights_stride = a.weights_stride;
  p.decay = a.decay;
  p.window = a.window;
  p.query_start = a.query_start;
  p.context_lens = a.context_lens;
  p.block_tables = a.block_tables;
  p.status = a.status;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.max_context_len = a.max_context_len;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.group_pow2 = 1;
  while (p.group_pow2 < p.group) p.group_pow2 <<= 1;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.total_queries = a.total_queries;
  p.qscale = a.scale * 1.4426950408889634f;
  p.key_tiles = (a.max_context_len + kKeys - 1) / kKeys;
  const long long ctas = (long long)p.key_tiles * a.num_kv_heads * a.num_seqs;
  CUtensorMap qm, km;
  const long long rows = (long long)a.num_blocks * a.num_kv_heads * a.block_size;
  if (ctas > 0x7fffffffLL ||
      !make_cache_map(&km, a.k_cache, a.dtype, rows, a.head_dim, a.block_size) ||
      !make_token_head_map(&qm, a.q, a.dtype, a.total_queries, a.num_q_heads, a.head_dim,
                           p.group_pow2, kRows / p.group_pow2)) {
    *unsupported = true;
    return cudaErrorInvalidValue;
  }
  if (a.dtype == PKV_F16)
    return a.head_dim == 64 ? launch_pw_typed<__half, 64>(p, qm, km, (int)ctas, stream)
                            : launch_pw_typed<__half, 128>(p, qm, km, (int)ctas, stream);
  return a.head_dim == 64 ? launch_pw_typed<__nv_bfloat16, 64>(p, qm, km, (int)ctas, stream)
                          : launch_pw_typed<__nv_bfloat16, 128>(p, qm, km, (int)ctas, stream);
}

}  // namespace pkv
