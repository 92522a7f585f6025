// Rotary positions fused with the append of new tokens: q rotated into q_out,
// k rotated into its cache slot, v copied into its slot, one pass over the
// projection's rows.
//
// Pair i < R / 2 of a head row (R = rotated dimensions) is turned by the angle
// position * inv_freq[i]:
//   a' = f (a cos - b sin),  b' = f (a sin + b cos)
// with (a, b) the elements (2 i, 2 i + 1) (interleaved) or (i, i + R / 2)
// (half); elements from R on pass through.  The angle is formed and reduced to
// one turn in 64 bits: at position 10^6 a 32-bit product would be off by 0.06
// radians.  The products are 32-bit and each result is rounded once, to the
// element type that q_out and the cache hold.
//
// Bound by HBM: (Hq + 2 Hkv) D elements read and as many written per token.

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;

enum RopeLayout { kInterleaved = 0, kHalf = 1, kHalfScalar = 2 };

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = a * cs.y + b * cs.x;
  a = x;
}

// Four pairs of neighbours in one 16-byte chunk: pairs p0 .. p0 + 3, those
// below `pairs` turned.
template <typename T>
__device__ __forceinline__ uint4 rotate_neighbours(uint4 w, const float2* cs, int p0, int pairs) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (p0 + j < pairs) {
      float2 x = Cvt<T>::to_float2(u[j]);
      rotate(x.x, x.y, cs[p0 + j]);
      u[j] = Cvt<T>::from_float2(x.x, x.y);
    }
  }
  return w;
}

// Eight pairs (p0 + j, p0 + j + R / 2): `lo` holds the first elements, `hi`
// the second.
template <typename T>
__device__ __forceinline__ void rotate_halves(uint4& lo, uint4& hi, const float2* cs, int p0) {
  uint32_t* ul = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* uh = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 a = Cvt<T>::to_float2(ul[j]), b = Cvt<T>::to_float2(uh[j]);
    rotate(a.x, b.x, cs[p0 + 2 * j]);
    rotate(a.y, b.y, cs[p0 + 2 * j + 1]);
    ul[j] = Cvt<T>::from_float2(a.x, a.y);
    uh[j] = Cvt<T>::from_float2(b.x, b.y);
  }
}

// Every unit of a head row (16 elements; two elements in the scalar layout)
// is read and written by one thread, reads first, so q_out may be q.
template <typename T, int LAYOUT>
__device__ __forceinline__ void rope_unit(const T* src, T* dst, int u, int rot, const float2* cs) {
  if constexpr (LAYOUT == kHalfScalar) {
    const int half = rot / 2;
    const int i = u < half ? u : 2 * u;          // past the pairs: elements R, R + 2, ...
    const int j = u < half ? u + half : 2 * u + 1;
    float a = static_cast<float>(src[i]), b = static_cast<float>(src[j]);
    if (u < half) rotate(a, b, cs[u]);
    dst[i] = static_cast<T>(a);
    dst[j] = static_cast<T>(b);
  } else {
    // chunks c0 and c1 of the row
    int c0 = 2 * u, c1 = 2 * u + 1;
    const bool turned = LAYOUT == kHalf && u < rot / 16;
    if (turned) {
      c0 = u;
      c1 = u + rot / 16;
    }
    uint4 x = reinterpret_cast<const uint4*>(src)[c0];
    uint4 y = reinterpret_cast<const uint4*>(src)[c1];
    if (turned) {
      rotate_halves<T>(x, y, cs, 8 * u);
    } else if (LAYOUT == kInterleaved) {
      x = rotate_neighbours<T>(x, cs, 4 * c0, rot / 2);
      y = rotate_neighbours<T>(y, cs, 4 * c1, rot / 2);
    }
    reinterpret_cast<uint4*>(dst)[c0] = x;
    reinterpret_cast<uint4*>(dst)[c1] = y;
  }
}

// One CTA per token.
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kv_append_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ float2 cs[64];  // (cos, sin) of each pair
  const int t = blockIdx.x;
  const int pos = p.positions[t];
  if (pos < 0) return;  // padding
  const int pairs = p.rot_dim / 2;
  if (threadIdx.x < pairs) {
    const double turns = (double)pos * (p.inv_freq[threadIdx.x] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[threadIdx.x] = make_float2(c * p.factor, s * p.factor);
  }
  const long long slot = p.slot_mapping[t];
  bool store = slot >= 0;
  if (slot >= p.num_slots) {
    if (threadIdx.x == 0) atomicOr(p.status, PKV_DEV_BAD_SLOT);
    store = false;
  }
  __syncthreads();
  const int D = p.head_dim;
  const long long blk = store ? slot / p.block_size : 0;
  const long long off = store ? slot - blk * p.block_size : 0;
  const int units = LAYOUT == kHalfScalar ? D / 2 : D / 16;
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  T* qo = static_cast<T*>(p.q_out) + t * p.q_out_stride;
  for (int i = threadIdx.x; i < p.num_q_heads * units; i += kRopeThreads) {
    const int h = i / units;
    rope_unit<T, LAYOUT>(q + h * D, qo + h * D, i - h * units, p.rot_dim, cs);
  }
  if (!store) return;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  T* kc = static_cast<T*>(p.k_cache);
  T* vc = static_cast<T*>(p.v_cache);
  const size_t row0 = (size_t)blk * p.num_kv_heads * p.block_size + off;
  for (int i = threadIdx.x; i < p.num_kv_heads * units; i += kRopeThreads) {
    const int h = i / units;
    rope_unit<T, LAYOUT>(k + h * D, kc + (row0 + (size_t)h * p.block_size) * D, i - h * units,
                         p.rot_dim, cs);
  }
  for (int i = threadIdx.x; i < p.num_kv_heads * (D / 8); i += kRopeThreads) {
    const int h = i / (D / 8), c = i - h * (D / 8);
    reinterpret_cast<uint4*>(vc + (row0 + (size_t)h * p.block_size) * D)[c] =
        reinterpret_cast<const uint4*>(v + h * D)[c];
  }
}

template <typename T>
cudaError_t launch_rope_typed(const RopeParams& p, int num_tokens, cudaStream_t stream) {
  const dim3 grid(num_tokens), block(kRopeThreads);
  if (p.interleaved)
    return launch_overlapped(rope_kv_append_kernel<T, kInterleaved>, grid, block, 0, stream, p);
  if (p.rot_dim % 16 == 0)
    return launch_overlapped(rope_kv_append_kernel<T, kHalf>, grid, block, 0, stream, p);
  return launch_overlapped(rope_kv_append_kernel<T, kHalfScalar>, grid, block, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeParams& p, int num_tokens, int dtype,
                                  cudaStream_t stream) {
  return dtype == PKV_F16 ? launch_rope_typed<__half>(p, num_tokens, stream)
                          : launch_rope_typed<__nv_bfloat16>(p, num_tokens, stream);
}

}  // namespace pkv
