// Norms of the query and key heads with rotary positions, in one pass:
//   y = x * w / sqrt(mean x^2 + eps)      (without weights: y = x)
// over each head row, then pair i < R / 2 of the row turned by the angle
// positions[axis(i)] * inv_freq[i], as rope_kv_append turns it.  The axes are
// those of a picture or a film (time, height, width), each of which turns its
// own pairs; text has one.
//
// The mean and the products are 32-bit, the angle is formed and reduced to one
// turn in 64 bits, and each element is rounded once, at the end.  Bound by HBM:
// (Hq + Hkv) D elements read and as many written per token: 16,384 tokens of 32 + 8
// heads of 128 with three axes 59.5 us, 5,640 GB/s.  (A CTA per token, sines and
// cosines read from shared memory for every head: 104; kept in registers, the next
// turn's rows in registers, too: 70; four turns ahead in shared memory: 58; two
// and three ahead 68 and 60, four CTAs per SM instead of three 68.)

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // most tokens per CTA

enum Layout { kInterleaved = 0, kHalf = 1, kHalfAny = 2 };

__device__ __forceinline__ void copy_async(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}

__device__ __forceinline__ Pair rotated(Pair v, float2 cs) {
  const float2 x = both(v);
  return pair(x.x * cs.x - x.y * cs.y, x.x * cs.y + x.y * cs.x);
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 w, Pair* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = Cvt<T>::to_float2(u[j]);
    f[j] = pair(x.x, x.y);
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const Pair* f) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = both(f[j]);
    u[j] = Cvt<T>::from_float2(x.x, x.y);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A unit is two 16-byte chunks of a head row; D / 16 neighbouring threads hold
// a row and add up its squares by shuffles.  The chunks are w and w + R / 16
// where those hold the two halves of the same pairs, else two that one thread
// can turn alone.  Halves that do not fill chunks (R not a multiple of 16) meet
// in shared memory.  Each element is read and written by one thread, so the
// outputs may be the inputs.
//
// The warps of a token go through its heads 512 / D at a time.  A thread's
// pairs and dimensions are the same in every head, so their sines, cosines and
// weights stay in registers.  The rows of the next turns are on their way into
// shared memory, each thread's own chunks, so that nothing waits on other warps.
template <typename T, int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads, 3)
    qk_norm_rope_kernel(const NormRopeParams p, int num_tokens, int tokens_per_cta) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  constexpr int kUpr = D / 16;       // units per head row
  constexpr int kHeads = 32 / kUpr;  // heads a warp works on at once
  constexpr int kDepth = LAYOUT == kHalfAny ? 2 : 4;  // turns of heads on their way
  __shared__ float2 cs[kTokens][64];
  __shared__ uint4 stages[kDepth][2][kThreads];
  __shared__ float rows[LAYOUT == kHalfAny ? kThreads / kUpr : 1][D + 1];
  const int t0 = blockIdx.x * tokens_per_cta;
  const int n = min(tokens_per_cta, num_tokens - t0);
  const int pairs = p.rot_dim / 2;
  // The first heads' rows are on their way while the angles are worked out.
  const int warps = kThreads / 32 / tokens_per_cta;  // of each token
  const int tok = (threadIdx.x >> 5) / warps, part = (threadIdx.x >> 5) % warps;
  const int lane = threadIdx.x & 31;
  const int turned = LAYOUT == kHalf ? p.rot_dim / 16 : 0;
  const int w = lane % kUpr;
  const int c0 = LAYOUT != kHalf || w < turned ? w : 2 * w;
  const int c1 = LAYOUT != kHalf ? w + kUpr : (w < turned ? w + turned : 2 * w + 1);
  const long long tt = t0 + tok;
  const bool real = tok < n && p.positions[tt] >= 0;
  // A turn of heads is of q or of k.
  const int q_turns = (p.num_q_heads + kHeads - 1) / kHeads;
  const int turns = q_turns + (p.num_kv_heads + kHeads - 1) / kHeads;
  auto head_of = [&](int turn) {
    return (turn < q_turns ? turn : turn - q_turns) * kHeads + lane / kUpr;
  };
  const T* q_row = static_cast<const T*>(p.q) + tt * p.q_stride;
  const T* k_row = static_cast<const T*>(p.k) + tt * p.k_stride;
  auto load = [&](int turn, int stage) {
    const int h = head_of(turn);
    const bool there =
        real && turn < turns && h < (turn < q_turns ? p.num_q_heads : p.num_kv_heads);
    if (there) {
      const uint4* row = reinterpret_cast<const uint4*>((turn < q_turns ? q_row : k_row) +
                                                        (long long)h * D);
      copy_async(&stages[stage][0][threadIdx.x], row + c0);
      copy_async(&stages[stage][1][threadIdx.x], row + c1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) load(part + i * warps, i);

  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int at = i / pairs, pair = i - at * pairs;
    const int pos = p.positions[(long long)p.pair_axes[pair] * p.positions_stride + t0 + at];
    const double turns = (double)pos * (p.inv_freq[pair] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[at][pair] = make_float2(c * p.factor, s * p.factor);
  }
  __syncthreads();
  if (!real) return;  // (whole warps)

  const float2* a = cs[tok];
  float2 mine[LAYOUT == kInterleaved ? 8 : 1];
  Pair c2[4], s2[4], n2[4];  // cosines, sines and minus the sines of two pairs
  if (LAYOUT == kInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mine[j] = a[j < 4 ? 4 * c0 + j : 4 * c1 + j - 4];
  } else if (LAYOUT == kHalf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = a[8 * w + 2 * j], v = a[8 * w + 2 * j + 1];
      c2[j] = pair(u.x, v.x);
      s2[j] = pair(u.y, v.y);
      n2[j] = pair(-u.y, -v.y);
    }
  }
  T* q_out = static_cast<T*>(p.q_out) + tt * p.q_out_stride;
  T* k_out = static_cast<T*>(p.k_out) + tt * p.k_out_stride;
  Pair wx[4], wy[4];  // the weights of this thread's dimensions, of q or of k
  const T* weights = nullptr;
  int stage = 0;
  for (int turn = part; turn < turns; turn += warps) {
    const bool is_q = turn < q_turns;
    const int h = head_of(turn);
    Pair x[4], y[4];
    load(turn + (kDepth - 1) * warps, (stage + kDepth - 1) % kDepth);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    unpack<T>(stages[stage][0][threadIdx.x], x);
    unpack<T>(stages[stage][1][threadIdx.x], y);
    stage = (stage + 1) % kDepth;
    const T* now = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    if (now) {
      if (now != weights) {
        weights = now;
        unpack<T>(__ldg(reinterpret_cast<const uint4*>(now) + c0), wx);
        unpack<T>(__ldg(reinterpret_cast<const uint4*>(now) + c1), wy);
      }
      Pair sq = pair(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) sq = fma2(x[j], x[j], fma2(y[j], y[j], sq));
      float sum = both(sq).x + both(sq).y;
#pragma unroll
      for (int mk = kUpr / 2; mk >= 1; mk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mk);
      float mean = sum * (1.f / D) + p.eps;
      // bf16 reaches squares that 32 bits do not hold: such a row is scaled by a power
      // of two first, eps with it.
      const bool held = mean >= 0x1p-100f && mean <= 0x1p+120f;
      if (std::is_same<T, __nv_bfloat16>::value && __any_sync(0xffffffffu, !held)) {
        float top = sqrtf(p.eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = both(x[j]), v = both(y[j]);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y))));
        }
#pragma unroll
        for (int mk = kUpr / 2; mk >= 1; mk >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, mk));
        // 2^-e of top = 1.m 2^e, within what a normal number holds; 1 for a row that is held
        const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
        const float by = held ? 1.f : __uint_as_float((254u - e) << 23);
        const Pair by2 = pair(by, by);
        sq = pair(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = mul2(x[j], by2);
          y[j] = mul2(y[j], by2);
          sq = fma2(x[j], x[j], fma2(y[j], y[j], sq));
        }
        sum = both(sq).x + both(sq).y;
#pragma unroll
        for (int mk = kUpr / 2; mk >= 1; mk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mk);
        mean = sum * (1.f / D) + p.eps * by * by;
      }
      const float r = rsqrtf(mean);
      const Pair r2 = pair(r, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = mul2(x[j], mul2(r2, wx[j]));
        y[j] = mul2(y[j], mul2(r2, wy[j]));
      }
    }
    if (LAYOUT == kInterleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * c0 + j < pairs) x[j] = rotated(x[j], mine[j]);
        if (4 * c1 + j < pairs) y[j] = rotated(y[j], mine[4 + j]);
      }
    } else if (LAYOUT == kHalf) {
      if (w < turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // as rotated() does it, two pairs at once
          const Pair t = fma2(x[j], c2[j], mul2(y[j], n2[j]));
          y[j] = fma2(x[j], s2[j], mul2(y[j], c2[j]));
          x[j] = t;
        }
      }
    } else {
      float* row = rows[threadIdx.x / kUpr];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = both(x[j]), v = both(y[j]);
        row[8 * c0 + 2 * j] = u.x;
        row[8 * c0 + 2 * j + 1] = u.y;
        row[8 * c1 + 2 * j] = v.x;
        row[8 * c1 + 2 * j + 1] = v.y;
      }
      __syncwarp();
      auto turned_at = [&](float v, int i) {  // the other element of the pair from its owner
        if (i >= p.rot_dim) return v;
        const float2 c = a[i < pairs ? i : i - pairs];
        return i < pairs ? v * c.x - row[i + pairs] * c.y : row[i - pairs] * c.y + v * c.x;
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = both(x[j]), v = both(y[j]);
        x[j] = pair(turned_at(u.x, 8 * c0 + 2 * j), turned_at(u.y, 8 * c0 + 2 * j + 1));
        y[j] = pair(turned_at(v.x, 8 * c1 + 2 * j), turned_at(v.y, 8 * c1 + 2 * j + 1));
      }
    }
    if (h >= (is_q ? p.num_q_heads : p.num_kv_heads)) continue;
    uint4* out = reinterpret_cast<uint4*>((is_q ? q_out : k_out) + (long long)h * D);
    out[c0] = pack<T>(x);
    out[c1] = pack<T>(y);
  }
}

template <typename T, int D>
cudaError_t launch_typed(const NormRopeParams& p, int num_tokens, int sms, cudaStream_t stream) {
  // Eight tokens per CTA share its sines and cosines evenly (four: 63 us instead of
  // 58 at 16,384 tokens); fewer where that would leave SMs without a CTA.
  int tokens = kTokens;
  while (tokens > 1 && num_tokens < 2 * sms * tokens) tokens /= 2;
  const dim3 grid((num_tokens + tokens - 1) / tokens), block(kThreads);
  if (p.interleaved)
    return launch_overlapped(qk_norm_rope_kernel<T, D, kInterleaved>, grid, block, 0, stream, p,
                             num_tokens, tokens);
  if (p.rot_dim % 16 == 0)
    return launch_overlapped(qk_norm_rope_kernel<T, D, kHalf>, grid, block, 0, stream, p,
                             num_tokens, tokens);
  return launch_overlapped(qk_norm_rope_kernel<T, D, kHalfAny>, grid, block, 0, stream, p,
                           num_tokens, tokens);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, int num_tokens, int head_dim, int dtype,
                                int sms, cudaStream_t stream) {
  if (dtype == PKV_F16)
    return head_dim == 64 ? launch_typed<__half, 64>(p, num_tokens, sms, stream)
                          : launch_typed<__half, 128>(p, num_tokens, sms, stream);
  return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, num_tokens, sms, stream)
                        : launch_typed<__nv_bfloat16, 128>(p, num_tokens, sms, stream);
}

}  // namespace pkv
