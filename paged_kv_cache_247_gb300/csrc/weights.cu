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

// ---- decode: split contexts -------------------------------------------------

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
  const int np = context_partitions(ctx, p.partition_size);
  if (np <= 1) return;  // done by the decode kernel
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
// One CTA per (KT 128-key tiles, KV head, sequence): S^T = K_tile . Q^T with the
// keys as the MMA's M dimension (one tensor-memory lane per key) and NR
// (query, head) rows as N, for every tile of query rows that sees the keys.
// A thread adds up its key's row of 2^(x - lse): no exchange between threads,
// no atomics, and the same order of additions whatever runs beside it.
//
//   KT * PP warpgroups  the sums, one thread per key: each key tile has PP of
//                       them, which take the query tiles in turn, each with
//                       an S^T buffer of its own
//   producer warp       the K tiles once, then the Q tiles into a ring
//   issuer warp         the products; owns the tensor memory
//   column warp         each Q tile's log-sums and positions into a ring
//
// What bounds it is the chain from one product to the next through four S^T
// buffers: a wait on a ready barrier takes a warp about 150 cycles, eight MMAs
// and their commit 700, the sums of 128 columns 1,900 with four warps per
// scheduler.  That is the price of one buffer per warpgroup (the four fill tensor
// memory): a warpgroup's sums and the product that refills its buffer alternate.
// On 8 chunks of 2,048 queries over contexts of 4,096 (32 heads over
// 8 of 128) the products alone would take 187 us (64 cycles per 128 x 128 x 16)
// and the exponentials 174 (32 a cycle and SM).  Measured: 628 us with KT = 1 and
// every product masked, 423 with masks only where some row does not see some key,
// 370 with KT = 2 (half the Q tiles per key); 290 of them remain with the sums
// left out.  Slower: K as an operand in tensor memory (three warpgroups 402,
// 96-row tiles 407), an issuer warp per key tile and asynchronous copies of the
// log-sums (395), a buffer given back once its last 64 columns are in registers
// (408).  Where a sequence has at most 32 rows per KV head (a short window),
// NR = 32, KT = 1 and one warpgroup leave room for four CTAs per SM, which hide
// each other's chain of latencies (16 prompts, 40 heads, window 32: 47 -> 27 us;
// 16 contexts of 4,096 over 8 KV heads, window 32: 43 us with single heads, 85 on
// 128-row tiles.  With groups of 2 and 4, above the limit, the 128-row tiles take
// 105 and 123 us and 32-row tiles would take 65 and 78; from 8 on the two tie).
// A group that is no power of two masks every tile: the same 8 chunks with groups
// of 3 and 7 spend 532 and 1,022 us here, with groups of 4 and 8 383 and 727.

constexpr int kKeys = kTileKeys;

// Wait for this thread's tensor-memory loads.  It names the loaded registers
// and nothing else, so that shared-memory reads may move across it (with a
// memory clobber each step of the sums began with their latency).
__device__ __forceinline__ void wait_columns(float* v) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
        "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
        "+f"(v[14]), "+f"(v[15]));
}

template <int D, int NR>
struct PwShape {
  static constexpr int KT = NR == 128 ? 2 : 1;
  static constexpr int PP = NR == 128 ? 2 : 1;
  static constexpr int WG = KT * PP;
  static constexpr int kSumThreads = 128 * WG;
  static constexpr int kProducerWarp = 4 * WG;
  static constexpr int kIssuerWarp = kProducerWarp + 1;
  static constexpr int kColumnWarp = kProducerWarp + 2;
  static constexpr int kThreads = kSumThreads + 96;
  static constexpr int kCtas = NR == 128 ? 1 : 4;  // per SM: what the registers are sized for
  static constexpr int kTmem = NR * WG;
  static constexpr int kGroup = (D / 64) * 1024;
  static constexpr int kKTile = (kKeys / 8) * kGroup;
  static constexpr int kQTile = (NR / 8) * kGroup;
  static constexpr int kStages = NR == 128 ? 4 : 2;
  static constexpr int kQ = KT * kKTile;
  static constexpr int kSlots = 4;                     // column ring
  static constexpr int kLse = kQ + kStages * kQTile;   // [kSlots][NR] negated log-sums
  static constexpr int kPos = kLse + kSlots * NR * 4;  // [kSlots][NR] positions, -1: no row
  static constexpr int kSum = kPos + kSlots * NR * 4;  // [KT][128] the second warpgroup's sums
  static constexpr int kBar = kSum + KT * kKeys * 4;
  static constexpr int kBars = 2 + 2 * kStages + 2 * WG + 2 * kSlots;
  static constexpr int kTmemSlot = kBar + kBars * 8;
  static constexpr int kBytes = kTmemSlot + 16 + 1024;  // + alignment slack
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory per SM");
  static_assert(kTmem <= 512, "tensor memory");
};

template <typename T, int D, int NR>
__global__ void __launch_bounds__(PwShape<D, NR>::kThreads, PwShape<D, NR>::kCtas)
    prefill_weights_kernel(const PrefillWeightsParams p, const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap) {
  using L = PwShape<D, NR>;
  constexpr int S = L::kStages, C = L::kSlots, KT = L::KT, PP = L::PP, WG = L::WG;
  grid_dep_wait();
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sK = smem;
  unsigned char* sQ = smem + L::kQ;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* drain = k_full + 1;
  uint64_t* q_full = drain + 1;     // [S] Q tile landed
  uint64_t* q_empty = q_full + S;   // [S] products done reading it (commit)
  uint64_t* s_full = q_empty + S;   // [WG] S^T buffer computed (commit)
  uint64_t* s_free = s_full + WG;   // [WG] S^T buffer read (its four warps)
  uint64_t* c_full = s_free + WG;   // [C] columns of a tile written
  uint64_t* c_empty = c_full + C;   // [C] read by every warpgroup of the tile
  float* lse_ring = reinterpret_cast<float*>(smem + L::kLse);
  int* pos_ring = reinterpret_cast<int*>(smem + L::kPos);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kt = blockIdx.x % p.key_tiles;
  const int pair = blockIdx.x / p.key_tiles;
  const int kvh = pair % p.num_kv_heads, s = pair / p.num_kv_heads;
  const int G = p.group, Gp = p.group_pow2, qpt = NR / Gp;

  const int q0 = p.query_start[s];
  const int nq = p.query_start[s + 1] - q0;
  int ctx = p.context_lens[s];
  const long long cap = min((long long)p.max_context_len,
                            (long long)p.max_blocks_per_seq * p.block_size);
  if (nq <= 0 || q0 < 0 || ctx < nq) return;  // (a context too short: flagged by the attention)
  if (ctx > cap) ctx = (int)cap;
  const int key0 = kt * KT * kKeys;
  if (key0 >= ctx) return;
  // Queries j_lo .. nq - 1 count and see the first key tile (the last query
  // sees every key of the context).
  const int first = p.window > 0 ? max(0, nq - p.window) : 0;
  const int j_lo = max(first, key0 - (ctx - nq));
  const int n_tiles = (nq - j_lo + qpt - 1) / qpt;
  // The first query tile that sees key tile k (n_tiles if the context ends
  // before it).
  auto first_tile = [&](int k) {
    const int key = key0 + k * kKeys;
    return key >= ctx ? n_tiles : max(0, key - (ctx - nq) - j_lo) / qpt;
  };

  // The first tile of parity r (tiles i with i % PP == r) among them.
  auto first_turn = [&](int k, int r) {
    const int f = first_tile(k);
    return f + (r - f % PP + PP) % PP;
  };

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int b = 0; b < WG; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
    }
    for (int i = 0; i < C; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], 4 * KT);
    }
    fence_barrier_init();
  }
  if (warp == L::kIssuerWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(L::kTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == L::kProducerWarp) {
    // ------------------------------------------------------------- producer
    const int B = p.block_size;
    const int R = B < kKeys ? B : kKeys;
    const int nseg = (min(ctx - key0, KT * kKeys) + R - 1) / R;  // runs of all the key tiles
    if (lane == 0) mbar_arrive_expect_tx(k_full, (uint32_t)nseg * R * D * (uint32_t)sizeof(T));
    __syncwarp();
    for (int g = lane; g < nseg; g += 32) {
      const int key = key0 + g * R;
      int phys = __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + key / B);
      if ((unsigned)phys >= (unsigned)p.num_blocks) phys = 0;  // flagged by the attention kernel
      tma_load_group(sK + g * (R / 8) * L::kGroup, &kmap,
                     ((phys * p.num_kv_heads + kvh) * B + key % B) / 8, k_full);
    }
    __syncwarp();
    int issued = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int st = i % S;
      if (i >= S && !mbar_wait_warp(&q_empty[st], ((i / S) - 1) & 1, p.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[st], L::kQTile);
        tma_load_token_heads(sQ + st * L::kQTile, &qmap, kvh * G, q0 + j_lo + i * qpt, &q_full[st]);
      }
      __syncwarp();
      issued = i + 1;
    }
    // Copies still in flight at exit (only after a timeout) land first.
    mbar_drain(k_full, 0);
    for (int i = issued > S ? issued - S : 0; i < issued; ++i)
      mbar_drain(&q_full[i % S], (i / S) & 1);
    __syncwarp();
  } else if (warp == L::kIssuerWarp) {
    // --------------------------------------------------------------- issuer
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t idesc = instr_desc(bf16, false, false, NR, kKeys);
    const uint32_t aK = smem_addr(sK), aQ = smem_addr(sQ);
    int from[KT], begin[KT][PP];  // the first tile of each key tile, and of each S^T buffer
#pragma unroll
    for (int b = 0; b < WG; ++b) {
      from[b / PP] = first_tile(b / PP);
      begin[b / PP][b % PP] = first_turn(b / PP, b % PP);
    }
    bool ok = mbar_wait_warp(k_full, 0, p.status);
    for (int i = 0; ok && i < n_tiles; ++i) {
      const int st = i % S;
      if (!mbar_wait_warp(&q_full[st], (i / S) & 1, p.status)) break;
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        if (i < from[k]) continue;
        const int b = k * PP + i % PP;
        const int turn = (i - (i % PP ? begin[k][PP - 1] : begin[k][0])) / PP;  // uses before it
        if (turn > 0 && !mbar_wait_warp(&s_free[b], (turn - 1) & 1, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_f16_ss_warp(
              tmem + b * NR,
              smem_desc(aK + k * L::kKTile + (ks / 4) * 1024 + (ks % 4) * 32, 16, L::kGroup),
              smem_desc(aQ + st * L::kQTile + (ks / 4) * (NR * 128) + (ks % 4) * 32, 16, 1024),
              idesc, ks > 0 ? 1u : 0u);
        mma_commit_warp(&s_full[b]);
      }
      if (ok) mma_commit_warp(&q_empty[st]);
    }
    mma_commit_warp(drain);
    mbar_drain(drain, 0);
    __syncwarp();
  } else if (warp == L::kColumnWarp) {
    // -------------------------------------------------------------- columns
    // Column c of a tile is query row j, head g of the group.
    for (int i = 0; i < n_tiles; ++i) {
      const int sl = i % C;
      float nl[NR / 32];
      int pos[NR / 32];
#pragma unroll
      for (int c = 0; c < NR / 32; ++c) {
        const int col = c * 32 + lane;
        const int j = j_lo + i * qpt + col / Gp, g = col % Gp;
        const bool there = j < nq && g < G && q0 + j < p.total_queries;
        nl[c] = there ? -__ldg(p.lse + (size_t)(q0 + j) * p.num_q_heads + kvh * G + g)
                      : -CUDART_INF_F;
        pos[c] = there ? ctx - nq + j : -1;
      }
      if (i >= C && !mbar_wait_warp(&c_empty[sl], ((i / C) - 1) & 1, p.status)) break;
#pragma unroll
      for (int c = 0; c < NR / 32; ++c) {
        lse_ring[sl * NR + c * 32 + lane] = nl[c];
        pos_ring[sl * NR + c * 32 + lane] = pos[c];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c_full[sl]);
    }
  } else {
    // ----------------------------------------------------------------- sums
    const int t = threadIdx.x & 127;
    const int wg = WG == 1 ? 0 : threadIdx.x >> 7;
    const int my_key0 = key0 + wg / PP * kKeys;
    const int key = my_key0 + t;
    const int begin = first_turn(wg / PP, wg % PP);
    const uint32_t s_cols = tmem + wg * NR + ((uint32_t)((warp & 3) * 32) << 16);
    const float qs = p.qscale;
    const float2 qs2 = make_float2(qs, qs);
    float acc = 0.f, lost = 0.f;  // compensated: the low part of the running sum
    bool ok = true;
    int turn = 0;  // this warpgroup's tiles so far
    for (int i = wg % PP; i < n_tiles; i += PP) {
      const int sl = i % C;
      if (ok && !mbar_wait_warp(&c_full[sl], (i / C) & 1, p.status)) ok = false;
      if (i < begin) {  // the tile's queries do not see these keys
        __syncwarp();
        if (lane == 0) mbar_arrive(&c_empty[sl]);
        continue;
      }
      const int j0 = j_lo + i * qpt;
      const float* s_lse = lse_ring + sl * NR;
      const int* s_pos = pos_ring + sl * NR;
      // Masked: keys past some query's position, rows past the sequence's last
      // query, or heads past the group (other heads' rows, finite or not).
      const bool masked = my_key0 + kKeys - 1 > ctx - nq + j0 || j0 + qpt > nq || G != Gp ||
                          q0 + j0 + qpt > p.total_queries;
      const int cols = min(qpt, nq - j0) * Gp;
      if (ok && !mbar_wait_warp(&s_full[wg], turn & 1, p.status)) ok = false;
      tc_fence_after();
      float sum = 0.f;
      if (!masked) {
        // 16 columns at a time, the next 16 on their way from tensor memory.
        float2 part[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) part[k] = make_float2(0.f, 0.f);
        float x[2][16];
        tmem_ld16f(s_cols, x[0]);
        wait_columns(x[0]);
#pragma unroll
        for (int c0 = 0; c0 < NR; c0 += 16) {
          float* v = x[c0 / 16 & 1];
          float* next = x[~(c0 / 16) & 1];
          if (c0 + 16 < NR) tmem_ld16f(s_cols + c0 + 16, next);
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(s_lse + c0 + c);
            float2 a = __ffma2_rn(make_float2(v[c], v[c + 1]), qs2, make_float2(n4.x, n4.y));
            float2 b = __ffma2_rn(make_float2(v[c + 2], v[c + 3]), qs2, make_float2(n4.z, n4.w));
            a.x = ex2(a.x);
            a.y = ex2(a.y);
            b.x = ex2(b.x);
            b.y = ex2(b.y);
            part[(c >> 1) & 3] = __fadd2_rn(part[(c >> 1) & 3], a);
            part[((c >> 1) + 1) & 3] = __fadd2_rn(part[((c >> 1) + 1) & 3], b);
          }
          if (c0 + 16 < NR) wait_columns(next);
        }
        const float2 y = __fadd2_rn(__fadd2_rn(part[0], part[1]), __fadd2_rn(part[2], part[3]));
        sum = y.x + y.y;
      } else {
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 32) {
          float x[32];
          tmem_ld32f(s_cols + c0, x);
          tmem_wait_ld_bind(x);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float e = ex2(fmaf(x[c], qs, s_lse[c0 + c]));
            part[c & 3] += key <= s_pos[c0 + c] ? e : 0.f;
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // one arrival per warp: they are served one after another
        mbar_arrive(&s_free[wg]);
        mbar_arrive(&c_empty[sl]);
      }
      ++turn;
      const float y = sum - lost;
      const float z = acc + y;
      lost = (z - acc) - y;
      acc = z;
    }
    if constexpr (PP == 2) {
      float* s_sum = reinterpret_cast<float*>(smem + L::kSum) + wg / PP * kKeys;
      if (wg % PP == 1) s_sum[t] = acc;
      named_barrier_sync(1 + WG + wg / PP, 256);
      if (wg % PP == 0) acc += s_sum[t];
      ok = ok && !timed_out(p.status);
    }
    if (ok && wg % PP == 0 && key < ctx) {
      float* w = p.weights + ((size_t)s * p.num_kv_heads + kvh) * p.weights_stride + key;
      *w = decayed(p.decay, *w, acc);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kIssuerWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(L::kTmem));
  }
}

template <typename T, int D, int NR>
cudaError_t launch_pw_typed(const PrefillWeightsParams& p, const CUtensorMap& qm,
                            const CUtensorMap& km, int ctas, cudaStream_t stream) {
  using L = PwShape<D, NR>;
  static unsigned long long configured = 0;  // bit per device ordinal (< 64)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    err = cudaFuncSetAttribute(prefill_weights_kernel<T, D, NR>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (err != cudaSuccess) return err;
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  return launch_overlapped(prefill_weights_kernel<T, D, NR>, dim3(ctas), dim3(L::kThreads),
                           L::kBytes, stream, p, qm, km);
}

template <typename T, int NR>
cudaError_t launch_pw(const PrefillWeightsParams& p, const CUtensorMap& qm, const CUtensorMap& km,
                      int head_dim, int ctas, cudaStream_t stream) {
  return head_dim == 64 ? launch_pw_typed<T, 64, NR>(p, qm, km, ctas, stream)
                        : launch_pw_typed<T, 128, NR>(p, qm, km, ctas, stream);
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeParams& p, cudaStream_t stream) {
  const dim3 grid((p.max_context_len + kDwSpan - 1) / kDwSpan, p.num_kv_heads, p.num_seqs);
  return launch_overlapped(decode_weights_kernel, grid, dim3(kDwThreads), 0, stream, p);
}

namespace {

int pow2_group(const PrefillArgs& a) {
  int g = 1;
  while (g < a.num_q_heads / a.num_kv_heads) g <<= 1;
  return g;
}

// Query rows per tile.
int tile_rows(const PrefillArgs& a) {
  const long long most = a.window > 0 ? std::min(a.window, a.max_query_len) : a.max_query_len;
  return most * pow2_group(a) <= 32 ? 32 : 128;
}

// CTAs per (sequence, KV head).
int key_tiles(const PrefillArgs& a) {
  const int keys = kKeys * (tile_rows(a) == 128 ? PwShape<128, 128>::KT : PwShape<128, 32>::KT);
  return (a.max_context_len + keys - 1) / keys;
}

}  // namespace

long long prefill_weights_ctas(const PrefillArgs& a) {
  return (long long)key_tiles(a) * a.num_kv_heads * a.num_seqs;
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
  p.group_pow2 = pow2_group(a);
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.total_queries = a.total_queries;
  p.qscale = a.scale * 1.4426950408889634f;
  const int nr = tile_rows(a);
  p.key_tiles = key_tiles(a);
  const long long ctas = prefill_weights_ctas(a);
  if (ctas == 0) return cudaSuccess;  // no sequence holds a position
  CUtensorMap qm, km;
  const long long rows = (long long)a.num_blocks * a.num_kv_heads * a.block_size;
  if (!make_cache_map(&km, a.k_cache, a.dtype, rows, a.head_dim, a.block_size) ||
      !make_token_head_map(&qm, a.q, a.dtype, a.total_queries, a.num_q_heads, a.head_dim,
                           p.group_pow2, nr / p.group_pow2)) {
    *unsupported = true;
    return cudaErrorInvalidValue;
  }
  if (a.dtype == PKV_F16)
    return nr == 32 ? launch_pw<__half, 32>(p, qm, km, a.head_dim, (int)ctas, stream)
                    : launch_pw<__half, 128>(p, qm, km, a.head_dim, (int)ctas, stream);
  return nr == 32 ? launch_pw<__nv_bfloat16, 32>(p, qm, km, a.head_dim, (int)ctas, stream)
                  : launch_pw<__nv_bfloat16, 128>(p, qm, km, a.head_dim, (int)ctas, stream);
}

}  // namespace pkv
