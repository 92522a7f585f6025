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

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnits = 2;   // units in flight per thread before the first is used
constexpr int kRopeTokens = 8;  // most tokens per CTA

enum RopeLayout { kInterleaved = 0, kHalf = 1 };

// Plain loads (q_out may be q), not kept in L1.
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

// What a CTA knows of its tokens: (cos, sin) of each pair, and where k and v
// go (row of head 0 in the caches, -1: nowhere).
struct RopeTokens {
  float2 cs[kRopeTokens][64];
  long long row0[kRopeTokens];
  int padding[kRopeTokens];
};

__device__ __forceinline__ void prepare_tokens(const RopeParams& p, RopeTokens& sm, int t0, int n) {
  const int pairs = p.rot_dim / 2;
  for (int i = threadIdx.x; i < n * pairs; i += blockDim.x) {
    const int tok = i / pairs, pair = i - tok * pairs;
    const double turns =
        (double)p.positions[t0 + tok] * (p.inv_freq[pair] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    sm.cs[tok][pair] = make_float2(c * p.factor, s * p.factor);
  }
  if (threadIdx.x < n) {
    const int t = t0 + threadIdx.x;
    const bool padding = p.positions[t] < 0;
    const long long slot = p.slot_mapping[t];
    long long row0 = -1;
    if (!padding && slot >= 0) {
      if (slot >= p.num_slots) {
        atomicOr(p.status, PKV_DEV_BAD_SLOT);
      } else {
        const long long blk = slot / p.block_size;
        row0 = blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size);
      }
    }
    sm.row0[threadIdx.x] = row0;
    sm.padding[threadIdx.x] = padding;
  }
}

// A unit is two 16-byte chunks of a head row of q, k or v: chunks w and w + R/16
// where they hold the two halves of the same pairs, else chunks that one thread
// can turn alone.  Each is read and written by one thread, so q_out may be q.
// A CTA takes as many tokens as give each thread kRopeUnits units, and issues
// those loads before it looks at positions and slots: the angles (64-bit
// arithmetic at a low rate, and a barrier) then overlap them.  (16,384 tokens,
// 32 + 2 x 8 heads of 128, whose units fill a CTA for each token: 78 us with the
// angles first, 68 us so.  4 + 2 heads of 64, eight tokens a CTA: 11.1 us, 17.1
// with one token; 48 heads of 64, two tokens a CTA: 40.9 us, 37.0 with one.)
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kv_append_kernel(const RopeParams p, int num_tokens, int tokens_per_cta) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ RopeTokens sm;
  const int t0 = blockIdx.x * tokens_per_cta;
  const int n = min(tokens_per_cta, num_tokens - t0);
  const int D = p.head_dim;
  const int upr = D / 16, log2_upr = D == 128 ? 3 : 2;  // units per head row
  const int units = (p.num_q_heads + 2 * p.num_kv_heads) * upr;
  const int total = n * units;
  const int turned = LAYOUT == kHalf ? p.rot_dim / 16 : 0;  // units with both halves of pairs

  auto chunk0 = [&](int w) { return w < turned || LAYOUT != kHalf ? w : 2 * w; };
  auto chunk1 = [&](int w) {
    return LAYOUT != kHalf ? w + upr : (w < turned ? w + turned : 2 * w + 1);
  };
  // Head row of unit u of token t.
  auto source = [&](int t, int h) {
    const long long tt = t0 + t;
    if (h < p.num_q_heads) return static_cast<const T*>(p.q) + tt * p.q_stride + (long long)h * D;
    h -= p.num_q_heads;
    if (h < p.num_kv_heads)
      return static_cast<const T*>(p.k) + tt * p.k_stride + (long long)h * D;
    return static_cast<const T*>(p.v) + tt * p.v_stride + (long long)(h - p.num_kv_heads) * D;
  };
  uint4 x[kRopeUnits], y[kRopeUnits];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
      const int g = base + i * blockDim.x + threadIdx.x;
      if (g >= total) continue;
      const int t = n == 1 ? 0 : g / units;
      const int u = g - t * units, w = u & (upr - 1);
      const uint4* src = reinterpret_cast<const uint4*>(source(t, u >> log2_upr));
      x[i] = load_once(src + chunk0(w));
      y[i] = load_once(src + chunk1(w));
    }
  };
  load(0);
  prepare_tokens(p, sm, t0, n);
  __syncthreads();
  for (int base = 0; base < total; base += kRopeUnits * blockDim.x) {
    if (base > 0) load(base);
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
      const int g = base + i * blockDim.x + threadIdx.x;
      if (g >= total) continue;
      const int t = n == 1 ? 0 : g / units;
      const int u = g - t * units, w = u & (upr - 1);
      int h = u >> log2_upr;
      const bool is_q = h < p.num_q_heads;
      const bool is_v = h >= p.num_q_heads + p.num_kv_heads;
      if (is_q ? sm.padding[t] != 0 : sm.row0[t] < 0) continue;
      if (!is_v) {
        const float2* cs = sm.cs[t];
        if (LAYOUT == kInterleaved) {
          x[i] = rotate_neighbours<T>(x[i], cs, 4 * chunk0(w), p.rot_dim / 2);
          y[i] = rotate_neighbours<T>(y[i], cs, 4 * chunk1(w), p.rot_dim / 2);
        } else if (w < turned) {
          rotate_halves<T>(x[i], y[i], cs, 8 * w);
        }
      }
      T* dst;
      if (is_q) {
        dst = static_cast<T*>(p.q_out) + (t0 + t) * p.q_out_stride + (long long)h * D;
      } else {
        h -= p.num_q_heads + (is_v ? p.num_kv_heads : 0);
        dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
              (sm.row0[t] + (long long)h * p.block_size) * D;
      }
      reinterpret_cast<uint4*>(dst)[chunk0(w)] = x[i];
      reinterpret_cast<uint4*>(dst)[chunk1(w)] = y[i];
    }
  }
}

// The half layout where R is not a multiple of 16, so that a pair's halves lie
// in chunks at different offsets: one pair of elements per thread.  One CTA per
// token.  Bound by its 2-byte accesses and the angles ahead of them: 16,384 tokens
// of 32 + 2 x 8 heads of 128 with R = 100 take 192 us (R = 96: 68), with heads of 64
// and R = 46 125 us (R = 48: 41); 64 tokens 4.8 us (2.9).  Kept simple: models rotate
// multiples of 16 in this layout, and the other layout takes any R at full speed.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kv_append_scalar_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  __shared__ RopeTokens sm;
  const int t = blockIdx.x;
  prepare_tokens(p, sm, t, 1);
  __syncthreads();
  if (sm.padding[0]) return;
  const int D = p.head_dim, half = p.rot_dim / 2;
  auto turn_rows = [&](const T* src, T* dst, long long dst_head, int heads) {
    for (int g = threadIdx.x; g < heads * (D / 2); g += kRopeThreads) {
      const int h = g / (D / 2), u = g - h * (D / 2);
      const int i = u < half ? u : 2 * u;  // past the pairs: elements R, R + 2, ...
      const int j = u < half ? u + half : 2 * u + 1;
      const T* row = src + (long long)h * D;
      T* to = dst + h * dst_head;
      float a = static_cast<float>(row[i]), b = static_cast<float>(row[j]);
      if (u < half) rotate(a, b, sm.cs[0][u]);
      to[i] = static_cast<T>(a);
      to[j] = static_cast<T>(b);
    }
  };
  turn_rows(static_cast<const T*>(p.q) + t * p.q_stride,
            static_cast<T*>(p.q_out) + t * p.q_out_stride, D, p.num_q_heads);
  if (sm.row0[0] < 0) return;
  const long long dst_head = (long long)p.block_size * D;
  turn_rows(static_cast<const T*>(p.k) + t * p.k_stride,
            static_cast<T*>(p.k_cache) + sm.row0[0] * D, dst_head, p.num_kv_heads);
  const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
  T* vc = static_cast<T*>(p.v_cache) + sm.row0[0] * D;
  for (int i = threadIdx.x; i < p.num_kv_heads * (D / 8); i += kRopeThreads) {
    const int h = i / (D / 8), c = i - h * (D / 8);
    reinterpret_cast<uint4*>(vc + h * dst_head)[c] = reinterpret_cast<const uint4*>(v + h * D)[c];
  }
}

template <typename T>
cudaError_t launch_rope_typed(const RopeParams& p, int num_tokens, cudaStream_t stream) {
  if (!p.interleaved && p.rot_dim % 16)
    return launch_overlapped(rope_kv_append_scalar_kernel<T>, dim3(num_tokens), dim3(kRopeThreads),
                             0, stream, p);
  const long long units = (p.num_q_heads + 2LL * p.num_kv_heads) * (p.head_dim / 16);
  const long long span = (long long)kRopeUnits * kRopeThreads;  // units of a full CTA
  // Several tokens per CTA only where there are CTAs to spare: a short launch
  // takes one CTA's chain of latencies however few tokens a CTA has.
  const int tokens = (int)std::max(
      1LL, std::min({(long long)kRopeTokens, span / units, (long long)num_tokens / 1024}));
  const long long want = (tokens * units + kRopeUnits - 1) / kRopeUnits;
  const int threads = (int)std::min<long long>(kRopeThreads, (want + 31) / 32 * 32);
  const dim3 grid((unsigned)(((long long)num_tokens + tokens - 1) / tokens));
  return p.interleaved ? launch_overlapped(rope_kv_append_kernel<T, kInterleaved>, grid,
                                           dim3(threads), 0, stream, p, num_tokens, tokens)
                       : launch_overlapped(rope_kv_append_kernel<T, kHalf>, grid, dim3(threads), 0,
                                           stream, p, num_tokens, tokens);
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeParams& p, int num_tokens, int dtype,
                                  cudaStream_t stream) {
  return dtype == PKV_F16 ? launch_rope_typed<__half>(p, num_tokens, stream)
                          : launch_rope_typed<__nv_bfloat16>(p, num_tokens, stream);
}

}  // namespace pkv
