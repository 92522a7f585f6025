// Attention over a paged cache held in 8 bits (the format: fp8.cuh): one query
// per sequence, or the queries of a tree of drafted tokens ("Only 20.4% of your
// KV cache held actual tokens", section "The page table, relocated into
// attention"; "Why the KV cache is the thing that limits your batch": a decode
// step's time is the bytes of the cache).
//
// One CTA per (query row, query head).  Each thread takes one key of a tile of
// 128, the running maximum and sum are kept for the whole CTA, and then thread
// d adds up dimension d of the tile's V rows.

#include <math_constants.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kKeys = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kKeys) attn_fp8_simple_kernel(const AttnFp8Params p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float q_row[D], weight[kKeys], red[2][4];
  __shared__ long long v_row[kKeys];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int row = blockIdx.x, h = blockIdx.y, kvh = h / p.group;

  // The sequence whose queries hold this row.
  int s = row, j = 0, count = 1;
  if (p.query_start) {
    s = -1;
    for (int i = 0; i < p.num_seqs; ++i)
      if (p.query_start[i] <= row && row < p.query_start[i + 1]) s = i;
    if (s < 0) return;
    j = row - p.query_start[s];
    count = p.query_start[s + 1] - p.query_start[s];
    if (count > p.max_query_len) {
      if (t == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
      count = p.max_query_len;
      if (j >= count) return;
    }
  }
  const long long cap =
      min((long long)p.max_context_len, (long long)p.max_blocks_per_seq * p.block_size);
  int ctx = p.context_lens[s];
  if (ctx < 0 || ctx > cap || (p.query_start && count > ctx)) {
    if (t == 0) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    ctx = ctx < 0 ? 0 : (ctx > cap ? (int)cap : ctx);
  }
  const int base = p.query_start ? max(ctx - count, 0) : ctx;
  const unsigned long long mask = p.query_start ? (unsigned long long)p.tree_masks[row] : 0;

  const T* q = static_cast<const T*>(p.q) + ((long long)row * p.num_q_heads + h) * D;
  if (t < D) q_row[t] = static_cast<float>(q[t]) * p.qscale;
  __syncthreads();
  float m = -CUDART_INF_F, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < ctx; k0 += kKeys) {
    const int pos = k0 + t;
    const bool seen = pos < ctx && (pos < base || (mask >> (pos - base)) & 1);
    float x = -CUDART_INF_F, vs = 0.f;
    v_row[t] = -1;
    if (seen) {
      int blk = p.block_tables[(long long)s * p.max_blocks_per_seq + pos / p.block_size];
      if ((unsigned)blk >= (unsigned)p.num_blocks) {
        atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
        blk = 0;
      }
      const long long r =
          ((long long)blk * p.num_kv_heads + kvh) * p.block_size + pos % p.block_size;
      const uint4* codes = reinterpret_cast<const uint4*>(p.k_cache) + r * (D / 16);
      float dot = 0.f;
      for (int c = 0; c < D / 16; ++c) {
        const uint4 w = codes[c];
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = decode2(u[i / 2] >> (16 * (i % 2)));
          dot += v.x * q_row[16 * c + 2 * i] + v.y * q_row[16 * c + 2 * i + 1];
        }
      }
      x = dot * scale_value(p.k_scales[r]);
      vs = scale_value(p.v_scales[r]);
      v_row[t] = r;
    }
    float mx = x;
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, mk));
    if (lane == 0) red[0][warp] = mx;
    __syncthreads();
    const float mn =
        fmaxf(m, fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3])));
    const float alpha = m == mn ? 1.f : exp2f(m - mn);
    const float e = seen ? exp2f(x - mn) : 0.f;
    weight[t] = e * vs;
    float sum = e;
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mk);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    l = l * alpha + (red[1][0] + red[1][1] + red[1][2] + red[1][3]);
    o *= alpha;
    m = mn;
    if (t < D)
      for (int i = 0; i < kKeys; ++i)
        if (v_row[i] >= 0)
          o += weight[i] *
               decode2(reinterpret_cast<const uint8_t*>(p.v_cache)[v_row[i] * D + t]).x;
    __syncthreads();
  }
  if (t < D)
    static_cast<T*>(p.out)[((long long)row * p.num_q_heads + h) * D + t] =
        static_cast<T>(l == 0.f ? 0.f : o / l);
}

template <typename T>
cudaError_t launch_typed(const AttnFp8Params& p, int head_dim, cudaStream_t stream) {
  const dim3 grid(p.total_queries, p.num_q_heads);
  return head_dim == 64
             ? launch_overlapped(attn_fp8_simple_kernel<T, 64>, grid, dim3(kKeys), 0, stream, p)
             : launch_overlapped(attn_fp8_simple_kernel<T, 128>, grid, dim3(kKeys), 0, stream, p);
}

}  // namespace

cudaError_t launch_attn_fp8(const AttnFp8Params& p, int head_dim, int dtype, int sms,
                            cudaStream_t stream, bool* unsupported) {
  *unsupported = false;
  return dtype == PKV_F16 ? launch_typed<__half>(p, head_dim, stream)
                          : launch_typed<__nv_bfloat16>(p, head_dim, stream);
}

}  // namespace pkv
