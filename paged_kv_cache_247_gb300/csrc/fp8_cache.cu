// Rows into and out of a cache held in 8 bits (the format: fp8.cuh).
//
// kv_append_fp8: each token's K and V rows quantised into their slot, as
// kv_append writes them in 16 bits ("Only 20.4% of your KV cache held actual
// tokens", section "Why the KV cache is the thing that limits your batch": the
// cache's bytes bound the batch).  block_read_fp8: whole blocks back into 16
// bits, for the prompt-chunk attention, which reads those.
//
// Both are bound by HBM: 2 D bytes on the 16-bit side and D + 2 on the other
// per row.  Append of 16,384 tokens of 8 heads of 128: 17.5 us, 5,780 GB/s (with 8
// elements per thread, whose 16-byte loads are contiguous over a warp, 20.9: the
// shuffles and addresses of twice the threads then fill 73 % of the issue slots).
// Blocks of 8 x 4,096 positions read back: 33.1 us, 6,120 GB/s (16 elements per
// thread, stores of 16 bytes at strides of 32: 36.3).

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// The 16 codes of one thread's part of a row that LANES neighbouring threads
// hold, and the row's scale.
template <typename T, int LANES>
__device__ __forceinline__ uint4 quantise(const uint4 x[2], uint16_t* scale) {
  uint32_t m = __vmaxu2(max_magnitude(x[0]), max_magnitude(x[1]));
#pragma unroll
  for (int mk = LANES / 2; mk >= 1; mk >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, mk));
  const uint32_t a = max(m & 0xffffu, m >> 16);
  if (a >= Magnitude<T>::kInf) {
    *scale = kNanScale;
    return make_uint4(0, 0, 0, 0);
  }
  const int e = row_exponent(Magnitude<T>::value(a));
  const float inv = pow2(-e);
  *scale = scale_bits(e);
  return make_uint4(encode4<T>(x[0].x, x[0].y, inv), encode4<T>(x[0].z, x[0].w, inv),
                    encode4<T>(x[1].x, x[1].y, inv), encode4<T>(x[1].z, x[1].w, inv));
}

// The (token, head, 16-element part) triples form one index space; D / 16
// neighbouring threads hold a row and agree on its largest magnitude by
// shuffles.  The data is loaded before the slot, whose latency then overlaps.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv_append_fp8_kernel(const AppendFp8Params p, unsigned total, unsigned row_parts) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int kLanes = D / 16;
  const unsigned i = blockIdx.x * (unsigned)kThreads + threadIdx.x;
  const bool there = i < total;
  const unsigned t = there ? i / row_parts : 0;
  const unsigned r = there ? i - t * row_parts : 0;
  const unsigned h = r / kLanes, c = r % kLanes;
  uint4 k[2] = {}, v[2] = {};
  long long slot = -1;
  if (there) {
    const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) +
                                                     (long long)t * p.k_stride + r * 16ll);
    const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) +
                                                     (long long)t * p.v_stride + r * 16ll);
    k[0] = load_once(ks);
    k[1] = load_once(ks + 1);
    v[0] = load_once(vs);
    v[1] = load_once(vs + 1);
    slot = p.slot_mapping[t];
  }
  uint16_t k_scale, v_scale;
  const uint4 kc = quantise<T, kLanes>(k, &k_scale);
  const uint4 vc = quantise<T, kLanes>(v, &v_scale);
  if (slot < 0) return;  // padding
  if (slot >= p.num_slots) {
    if (r == 0) atomicOr(p.status, PKV_DEV_BAD_SLOT);
    return;
  }
  const long long blk = slot / p.block_size;
  const long long row =
      (blk * p.num_kv_heads + h) * p.block_size + (slot - blk * p.block_size);
  reinterpret_cast<uint4*>(p.k_cache)[row * kLanes + c] = kc;
  reinterpret_cast<uint4*>(p.v_cache)[row * kLanes + c] = vc;
  if (c == 0) {
    p.k_scales[row] = k_scale;
    p.v_scales[row] = v_scale;
  }
}

// Eight codes times the row's scale, rounded once to T (bf16 holds every
// product of a normal size exactly).
template <typename T>
__device__ __forceinline__ uint4 widen(uint2 codes, float scale) {
  const float2 a = decode2(codes.x), b = decode2(codes.x >> 16), c = decode2(codes.y),
               d = decode2(codes.y >> 16);
  return make_uint4(Cvt<T>::from_float2(a.x * scale, a.y * scale),
                    Cvt<T>::from_float2(b.x * scale, b.y * scale),
                    Cvt<T>::from_float2(c.x * scale, c.y * scale),
                    Cvt<T>::from_float2(d.x * scale, d.y * scale));
}

__device__ __forceinline__ uint2 load_once2(const uint2* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(p));
  return r;
}

// The (pair, 16-element part of the block) pairs form one index space, two
// threads to a part, so that a warp's 8-byte loads and 16-byte stores are
// contiguous.  A thread takes kEach shares and has all their loads on the way
// before the first is used.
constexpr int kEach = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    block_read_fp8_kernel(const ReadFp8Params p, unsigned total, unsigned block_parts) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int kParts = D / 16;  // of a row
  const unsigned half = threadIdx.x % 2;
  uint2 k[kEach], v[kEach];
  uint16_t ks[kEach], vs[kEach];
  long long to[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const unsigned i = (blockIdx.x * kEach + u) * (unsigned)(kThreads / 2) + threadIdx.x / 2;
    to[u] = -1;
    if (i >= total) continue;
    const unsigned pair = i / block_parts, c = i - pair * block_parts;
    const long long src = p.pairs[2ll * pair], dst = p.pairs[2ll * pair + 1];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_out_blocks) {
      if (c == 0) atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
      continue;
    }
    const long long from = src * block_parts + c;
    to[u] = 2 * (dst * block_parts + c) + half;
    k[u] = load_once2(reinterpret_cast<const uint2*>(p.k_cache) + 2 * from + half);
    v[u] = load_once2(reinterpret_cast<const uint2*>(p.v_cache) + 2 * from + half);
    ks[u] = p.k_scales[from / kParts];
    vs[u] = p.v_scales[from / kParts];
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    if (to[u] < 0) continue;
    reinterpret_cast<uint4*>(p.k_out)[to[u]] = widen<T>(k[u], scale_value(ks[u]));
    reinterpret_cast<uint4*>(p.v_out)[to[u]] = widen<T>(v[u], scale_value(vs[u]));
  }
}

template <typename T, int D>
cudaError_t append_typed(const AppendFp8Params& p, int num_tokens, cudaStream_t stream) {
  const long long parts = (long long)p.num_kv_heads * (D / 16), total = num_tokens * parts;
  return launch_overlapped(kv_append_fp8_kernel<T, D>,
                           dim3((unsigned)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           stream, p, (unsigned)total, (unsigned)parts);
}

template <typename T, int D>
cudaError_t read_typed(const ReadFp8Params& p, long long num_pairs, cudaStream_t stream) {
  const long long parts = (long long)p.num_kv_heads * p.block_size * (D / 16);
  const long long total = num_pairs * parts;
  constexpr int kPer = kThreads / 2 * kEach;
  return launch_overlapped(block_read_fp8_kernel<T, D>,
                           dim3((unsigned)((total + kPer - 1) / kPer)), dim3(kThreads), 0, stream,
                           p, (unsigned)total, (unsigned)parts);
}

}  // namespace

cudaError_t launch_kv_append_fp8(const AppendFp8Params& p, int num_tokens, int head_dim, int dtype,
                                 cudaStream_t stream) {
  if (dtype == PKV_F16)
    return head_dim == 64 ? append_typed<__half, 64>(p, num_tokens, stream)
                          : append_typed<__half, 128>(p, num_tokens, stream);
  return head_dim == 64 ? append_typed<__nv_bfloat16, 64>(p, num_tokens, stream)
                        : append_typed<__nv_bfloat16, 128>(p, num_tokens, stream);
}

cudaError_t launch_block_read_fp8(const ReadFp8Params& p, long long num_pairs, int head_dim,
                                  int dtype, cudaStream_t stream) {
  if (dtype == PKV_F16)
    return head_dim == 64 ? read_typed<__half, 64>(p, num_pairs, stream)
                          : read_typed<__half, 128>(p, num_pairs, stream);
  return head_dim == 64 ? read_typed<__nv_bfloat16, 64>(p, num_pairs, stream)
                        : read_typed<__nv_bfloat16, 128>(p, num_pairs, stream);
}

}  // namespace pkv
