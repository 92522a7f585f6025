// Norms of the query and key heads with rotary positions, in one pass:
//   y = x * w / sqrt(mean x^2 + eps)      (without weights: y = x)
// over each head row, then pair i < R / 2 of the row turned by the angle
// positions[axis(i)] * inv_freq[i], as rope_kv_append turns it.  The axes are
// those of a picture or a film (time, height, width), each of which turns its
// own pairs; text has one.
//
// The mean and the products are 32-bit, the angle is formed and reduced to one
// turn in 64 bits, and each element is rounded once, at the end.  Bound by HBM:
// (Hq + Hkv) D elements read and as many written per token.

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // most tokens per CTA

enum Layout { kInterleaved = 0, kHalf = 1, kHalfAny = 2 };

// Plain loads (the outputs may be the inputs), not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = a * cs.y + b * cs.x;
  a = x;
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = Cvt<T>::to_float2(u[j]);
    f[2 * j] = x.x;
    f[2 * j + 1] = x.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(Cvt<T>::from_float2(f[0], f[1]), Cvt<T>::from_float2(f[2], f[3]),
                    Cvt<T>::from_float2(f[4], f[5]), Cvt<T>::from_float2(f[6], f[7]));
}

// A unit is two 16-byte chunks of a head row; D / 16 neighbouring threads hold
// a row and add up its squares by shuffles.  The chunks are w and w + R / 16
// where those hold the two halves of the same pairs, else two that one thread
// can turn alone.  Halves that do not fill chunks (R not a multiple of 16) meet
// in shared memory.  Each element is read and written by one thread, so the
// outputs may be the inputs.
template <typename T, int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads)
    qk_norm_rope_kernel(const NormRopeParams p, int num_tokens, int tokens_per_cta) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int kUpr = D / 16;  // units per head row
  __shared__ float2 cs[kTokens][64];
  __shared__ int padding[kTokens];
  __shared__ float rows[LAYOUT == kHalfAny ? kThreads / kUpr : 1][D + 1];
  const int t0 = blockIdx.x * tokens_per_cta;
  const int n = min(tokens_per_cta, num_tokens - t0);
  const int pairs = p.rot_dim / 2;
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int tok = i / pairs, pair = i - tok * pairs;
    const int pos = p.positions[(long long)p.pair_axes[pair] * p.positions_stride + t0 + tok];
    const double turns = (double)pos * (p.inv_freq[pair] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[tok][pair] = make_float2(c * p.factor, s * p.factor);
  }
  if (threadIdx.x < n) padding[threadIdx.x] = p.positions[t0 + threadIdx.x] < 0;
  __syncthreads();

  const int heads = p.num_q_heads + p.num_kv_heads;
  const int units = heads * kUpr, total = n * units;
  const int turned = LAYOUT == kHalf ? p.rot_dim / 16 : 0;
  const int w = threadIdx.x % kUpr;
  const int c0 = LAYOUT != kHalf || w < turned ? w : 2 * w;
  const int c1 = LAYOUT != kHalf ? w + kUpr : (w < turned ? w + turned : 2 * w + 1);
  for (int base = 0; base < total; base += kThreads) {
    const int g = base + threadIdx.x;
    const bool there = g < total;
    const int t = there ? g / units : 0;
    const int h = there ? (g - t * units) / kUpr : 0;
    const bool is_q = h < p.num_q_heads;
    const int hh = is_q ? h : h - p.num_q_heads;
    const long long tt = t0 + t;
    float x[8], y[8];
    if (there) {
      const T* row = static_cast<const T*>(is_q ? p.q : p.k) +
                     tt * (is_q ? p.q_stride : p.k_stride) + (long long)hh * D;
      unpack<T>(load_once(reinterpret_cast<const uint4*>(row) + c0), x);
      unpack<T>(load_once(reinterpret_cast<const uint4*>(row) + c1), y);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
    }
    const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += x[j] * x[j] + y[j] * y[j];
#pragma unroll
    for (int mk = kUpr / 2; mk >= 1; mk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mk);
    if (weight) {
      const float r = rsqrtf(sum * (1.f / D) + p.eps);
      float wx[8], wy[8];
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(weight) + c0), wx);
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(weight) + c1), wy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] *= r * wx[j];
        y[j] *= r * wy[j];
      }
    }
    const float2* a = cs[t];
    if (LAYOUT == kInterleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * c0 + j < pairs) rotate(x[2 * j], x[2 * j + 1], a[4 * c0 + j]);
        if (4 * c1 + j < pairs) rotate(y[2 * j], y[2 * j + 1], a[4 * c1 + j]);
      }
    } else if (LAYOUT == kHalf) {
      if (w < turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rotate(x[j], y[j], a[8 * w + j]);
      }
    } else {
      float* row = rows[threadIdx.x / kUpr];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        row[8 * c0 + j] = x[j];
        row[8 * c1 + j] = y[j];
      }
      __syncwarp();
      auto turn = [&](float v, int i) {  // element i < R of its pair, the other from its owner
        const float2 c = a[i < pairs ? i : i - pairs];
        return i < pairs ? v * c.x - row[i + pairs] * c.y : row[i - pairs] * c.y + v * c.x;
      };
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (8 * c0 + j < p.rot_dim) x[j] = turn(x[j], 8 * c0 + j);
        if (8 * c1 + j < p.rot_dim) y[j] = turn(y[j], 8 * c1 + j);
      }
    }
    if (!there || padding[t]) continue;
    T* out = static_cast<T*>(is_q ? p.q_out : p.k_out) +
             tt * (is_q ? p.q_out_stride : p.k_out_stride) + (long long)hh * D;
    reinterpret_cast<uint4*>(out)[c0] = pack<T>(x);
    reinterpret_cast<uint4*>(out)[c1] = pack<T>(y);
  }
}

template <typename T, int D>
cudaError_t launch_typed(const NormRopeParams& p, int num_tokens, cudaStream_t stream) {
  const dim3 grid(num_tokens), block(kThreads);
  if (p.interleaved)
    return launch_overlapped(qk_norm_rope_kernel<T, D, kInterleaved>, grid, block, 0, stream, p,
                             num_tokens, 1);
  if (p.rot_dim % 16 == 0)
    return launch_overlapped(qk_norm_rope_kernel<T, D, kHalf>, grid, block, 0, stream, p,
                             num_tokens, 1);
  return launch_overlapped(qk_norm_rope_kernel<T, D, kHalfAny>, grid, block, 0, stream, p,
                           num_tokens, 1);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, int num_tokens, int head_dim, int dtype,
                                cudaStream_t stream) {
  if (dtype == PKV_F16)
    return head_dim == 64 ? launch_typed<__half, 64>(p, num_tokens, stream)
                          : launch_typed<__half, 128>(p, num_tokens, stream);
  return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, num_tokens, stream)
                        : launch_typed<__nv_bfloat16, 128>(p, num_tokens, stream);
}

}  // namespace pkv
