// Attention over a paged cache held in 8 bits (the format: fp8.cuh): one query
// per sequence, or the queries of a tree of drafted tokens ("Only 20.4% of your
// KV cache held actual tokens", section "The page table, relocated into
// attention"; section "Why the KV cache is the thing that limits your batch": a
// decode step's time is the bytes of the cache, here half of the 16-bit ones).
//
// The codes go from HBM through shared memory into the tensor core as they are
// (tcgen05.mma kind::f8f6f4); nothing is widened on the way.  The operands on
// the other side are split into 8-bit parts instead, which cost only columns of
// an N that is far from full:
//
//   q row      = 2^e (c1 + c2 / 16 + c3 / 256), e4m3 parts of 4 bits each, 2^e
//                as for a cache row: multiples of 2^(e - 17).  That is all of a
//                bf16 element from 2^-17 of the row's largest on, of an fp16 one
//                from 2^-14 on, and 2^-25 of the largest off at most for others.
//                (bf16 rows in two parts: from 2^-14 on, and 2^-21, and no faster:
//                32 x 4,096, 8 heads of 64 rows 106.2 us against 106.4 with three, of
//                32 rows 81.9 and 81.9, 4 heads of 16 rows 45.7 and 47.1, 64 x 8,192,
//                8 heads of 4 rows 186.4 and 184.3, each with the L2 cache flushed;)
//   S^T        [128 keys x parts * rows] = K codes . parts^T
//   x          = scale log2(e) 2^e k_scale (s1 + s2 / 16 + s3 / 256)
//   y          = x + lv, lv = log2 v_scale - E: the V row's scale, relative to a
//                reference 2^E, is an addend of the base-2 logit, and the running
//                reference m is one of y, which is what gets rounded: p =
//                2^(y - m) <= 2^15, to fp16, which is c1 + c2 / 16 + c3 / 256 in
//                e5m2: what each part leaves of 11 bits fits the next (3 bits and
//                twice 3 and the sign; at most 2^15), down to fp16's own smallest
//                step, 2^-24
//   O^T        [D x parts * rows] += V codes^T . parts
//   l          += p / 2^lv
//   out        = 2^E (o1 + o2 / 16 + o3 / 256) / l
//
// m moves when some y is 15 above it, to 6 below that y: half a step is at most
// 2^-31 of the largest p, and the largest has room to grow by 2^9 before m moves
// again, which costs about as much as a tile.  (Room for 2^12, 2^7 and 2^4, half a
// step of 2^-28, 2^-33 and 2^-36: 32 x 4,096, 8 heads of 64 rows 106.5, 112.3 and
// 117.4 us for 109.2, L2 flushed; decode the same.)
//
// lv is kept within -6 and 1, so that of a softmax weight at most 2^-31 2^7 = 2^-24
// of the largest is lost (2^-31 where the V rows' scales are the same), n times that
// over n positions at most, since l counts what they lose.  E is the largest scale
// of the item's first tile, and moves to a later tile's if that is more than twice
// as large; the O^T so far shrinks by as much.  Rows below 2^-6 of it are added
// apart, to an O^T of their own, in fp32 with their whole weights, and rows of zeros
// not at all.  That takes 0.6 us a tile for 4 rows, 3.4 for 64; where one token's V
// is small in each context, a call takes 0 to 6 % more.  That the code is there
// costs 64 rows 3 % and 4 nothing.  What is below 2^-126 of the largest row that
// some query of the item sees may be lost.
//
// Orientation, pipeline and roles follow the 16-bit decode kernel: keys are the
// first product's M, the D dimensions the second's (D = 64: an M of 64, whose
// row i lies in tensor-memory lane 32 (i / 16) + i % 16).  A work item is
// (sequence, KV head, partition of the context, up to 64 rows), a row being a
// query head of the group and one of the sequence's queries.  Two CTAs per SM (one
// from 33 rows on) go through the items; their rings, barriers and tensor memory
// flow from item to item, and an SM whose items are short takes more of them:
// the launch has a CTA per item, and where the device does not hold all of them a
// running one takes over those that have not started.  Warps:
//
//   key warpgroups (one; two and four, each with 16 rows, for more than 16 and 32):
//              thread t has key t of the tile: scales, logits, weights, and at
//              the end dimension t of the output.  Its parts of the weights are
//              neighbouring bytes (MN-major operand, no swizzle): one 16-byte
//              store for every 16 of them.
//   K, V producers   one TMA copy per (block, head) run into a ring of tiles, the
//              K warp also the scales of both
//   Q warps          rows split into their parts, an item ahead
//   item warp        the next items, from the CTAs that have not started
//   S, O issuers     four (D = 64: two, four) MMAs per tile
//
// Up to 8 rows the time is the cache's bytes: 64 x 8,192 positions, 8 heads of 128
// with 4 rows 161 us, 6,780 GB/s; 64 contexts of 16-2,048, 40 heads of one row 70 us,
// 5,370 GB/s, where the ends of items show.  More rows are bound by the key warps:
// 32 x 4,096, 8 heads of 64 rows 109 us, 2,560 GB/s, issue slots 56 % used where an
// SM works: 26 instructions a row and key warp for each tile, 4 of them the split in
// three.  What it took, at those three cases (us):
//   CUDA cores                                              2,406    349   3,998
//   this form, one CTA per SM, items dealt out beforehand     201    127     392
//   two floats per instruction, masks only in the last tiles  201    120     242
//   two CTAs per SM, items taken as they come, seldom code
//     kept short (met for the first time it runs at the
//     latency of its fetch)                                   164     76     165
//   weights in e5m2, one arrival per warp                     170     83     154
//   two CTAs per SM with two key warpgroups each              156     70     125
//   four key warpgroups: each tile once for 64 rows           161     69     100
//   three parts of bf16 queries, weights to 2^-31 of the
//     largest, V rows of any sizes                            161     70     109

#include <math_constants.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "overlap.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kKeys = kTileKeys;  // keys per tile
constexpr int kQParts = 3;        // e4m3 parts of a query row
constexpr int kParts = 3;         // e5m2 parts of a softmax weight
constexpr int kBufs = 2;          // buffers of the weights
constexpr int kItemBufs = 1;      // items handed out ahead (2 and 4: 64 short requests 1 and 4 us slower)
constexpr int kMostCtas = 8192;
constexpr float kExceed = 15.f;   // weights reach 2^15 before the reference moves,
constexpr float kPlace = 6.f;     // to where the largest is 2^6
constexpr float kStep = 16.f;     // what a part of a weight or a query leaves comes 16 times as large
constexpr float kNoRef = -3e38f;  // the reference of a row that saw nothing
// V scales are taken relative to a reference 2^E: rows from 2^(E - kBelow) to
// 2^(E + kAbove) go into the second product, smaller ones are added apart, larger
// ones move E.  E is held as the bits of the bfloat16 number 2^(E - kBelow).
constexpr int kAbove = 1, kBelow = 6;
constexpr int kBand = (kAbove + kBelow) * 128;
constexpr int kNoScale = 0x10000;  // before any: no scale's bits are in its band

// E of the scale with the given bits (no lower than 2^-120: a band that leaves out a
// scale of zero).
__device__ __forceinline__ int reference_of(int bits) { return max(bits - kBelow * 128, 0x80); }

// Registers with several key warpgroups.  Two: 256 threads of 96 and 256 of 32, out
// of 512 of 64 (88 and 40: 32 x 4,096, 8 heads of 32 rows 77.9 us for 71.6, L2
// flushed).  Four: 512 of 96 and 256 of 40, out of 768 of 80 (104 and 32: the same
// for 64 rows, and items of three tiles, whose starts the other warps' spills
// delay, 40 x 5,422, 5 heads of 34 rows 220 us for 200).
constexpr int kKeyRegs = 96;
constexpr int few_regs(int warpgroups) { return warpgroups == 2 ? 32 : 40; }

constexpr int up16(int x) { return (x + 15) / 16 * 16; }
constexpr int pow2_at_least(int x, int p = 32) { return p >= x ? p : pow2_at_least(x, 2 * p); }

template <int NH, int D>
struct Shape {
  static constexpr int NS = up16(kQParts * NH);  // columns of S^T
  static constexpr int NO = up16(kParts * NH);   // columns of O^T
  static constexpr int KG = NH > 16 ? NH / 16 : 1;  // key warpgroups
  static constexpr int NHW = NH / KG;               // rows per key warpgroup
  static constexpr int kPerSm = KG == 4 ? 1 : 2;    // CTAs per SM
  static constexpr int kQWarps = KG == 1 ? 1 : 2;
  static constexpr bool kKeysSplit = KG > 1;        // the first item's rows: see there
  // items' parts of q held, and buffers of S^T
  static constexpr int kQBufs = KG == 2 ? 1 : 2;
  static constexpr int SB = KG >= 2 ? 1 : 2;
  static constexpr int kKWarp = 4 * KG;
  static constexpr int kVWarp = kKWarp + 1;
  static constexpr int kSWarp = kKWarp + 2;  // owns tensor memory
  static constexpr int kOWarp = kKWarp + 3;
  static constexpr int kItemWarp = kKWarp + 4;
  static constexpr int kQWarp = kKWarp + 5;
  static constexpr int kReaders = kQWarp + kQWarps - 1;  // warps that read the items
  // Several key warpgroups take most of the registers, which warpgroups give
  // and take as a whole: one warp more, idle, fills the last.
  static constexpr int kWarps = KG == 1 ? kQWarp + kQWarps : 4 * KG + 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTile = kKeys * D;     // bytes of a K or V tile
  static constexpr int kQBytes = NS * D;
  static constexpr int kRawRows = NH < 16 ? NH : 16;
  static constexpr int kRaw = kRawRows * D * 2;  // q rows as they are, some at a time
  static constexpr int kPBuf = kKeys * NO;
  // scales, an item's rows, reductions, items, barriers; alignment
  static constexpr int kMaxStages = (KG == 2 ? 256 : KG == 4 ? 512 : 384) / D;  // (no more fit)
  static constexpr int kSmall = (kMaxStages + SB) * kKeys * 4 + 2 * NH * 16 + 5 * 4 * NH * 4 + 1024;
  static constexpr int kFixed = kQBufs * kQBytes + kRaw + kBufs * kPBuf + kSmall + 1024;
  static constexpr int kRoom = (kPerSm == 1 ? 227 : 113) * 1024;
  static constexpr int kFit = (kRoom - kFixed) / (2 * kTile);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kQ = 2 * kStages * kTile;  // after the K and V rings
  static constexpr int kQRaw = kQ + kQBufs * kQBytes;
  static constexpr int kP = kQRaw + kRaw;
  // A tile's scales come with its K rows.  Nothing says when they have been
  // read: they are before the tile's S^T is given back, without which the tile
  // SB later is not multiplied, without which its K stage does not get free.
  static constexpr int kScaleStages = kStages + SB;
  static constexpr int kScales = kP + kBufs * kPBuf;            // [stages][K, V][128] bfloat16
  static constexpr int kMasks = kScales + kScaleStages * kKeys * 4;  // [2][NH] 64-bit
  static constexpr int kFactors = kMasks + 2 * NH * 8;          // [2][NH] floats
  static constexpr int kRows = kFactors + 2 * NH * 4;           // [2][NH] output rows
  static constexpr int kTop = kRows + 2 * NH * 4;               // [KG][4 warps][NHW] floats
  static constexpr int kSum = kTop + 4 * NH * 4;                // [KG][4 warps][NHW]
  static constexpr int kRef = kSum + 4 * NH * 4;                // [KG][4 warps][NHW]
  static constexpr int kAlpha = kRef + 4 * NH * 4;              // [KG][4 warps][NHW]
  static constexpr int kShift = kAlpha + 4 * NH * 4;            // [KG][4 warps][NHW]
  static constexpr int kMarks = kShift + 4 * NH * 4;            // [KG][4 warps] integers
  static constexpr int kItems = kMarks + KG * 16;               // [kItemBufs] Item
  static constexpr int kTicket = kItems + kItemBufs * 64;
  static constexpr int kBar = kTicket + 16;
  static constexpr int kBars =
      4 * kStages + 2 * SB + 2 * kBufs + kScaleStages + 2 * kQBufs + 6 + 2 * kItemBufs + 2;
  static constexpr int kTmemSlot = kBar + kBars * 8;
  static constexpr int kBytes = kTmemSlot + 16 + 1024;
  static_assert(KG * 16 + kItemBufs * 64 + kBars * 8 + 32 <= 1024 && kBytes <= kRoom &&
                    kStages >= 2,
                "shared memory overflow");
  static constexpr int kColO = SB * NS;
  static constexpr int kColFar = kColO + NO;  // O^T of the V rows added apart
  static constexpr int kTmemCols = pow2_at_least(kColFar + NH);
  static_assert(kTmemCols <= 512 / kPerSm, "tensor memory overflow");
  static constexpr int kSwizzle = D == 128 ? 2 : 4;  // descriptor code of the D-byte swizzle
};

// Shared-memory matrix descriptor (version 1) with the given swizzle code.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lbo, uint32_t sbo, int swizzle) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)swizzle << 61);
}

// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bit 4), e4m3 codes
// of the cache times e4m3 parts of queries, both K-major, or e5m2 parts of
// weights (bits 10-12), both MN-major (bits 15, 16).
__device__ __forceinline__ uint32_t instr(bool weights, int n, int m) {
  return (1u << 4) | (weights ? 1u << 10 | 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// Warp-collective, as the helpers of tcgen05.cuh.
__device__ __forceinline__ void mma_f8_warp(uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// Offset of byte x of row r in rows of D bytes with the D-byte swizzle.
template <int D>
__device__ __forceinline__ int swizzled(int r, int x) {
  const int off = r * D + x;
  return off ^ (((off >> 7) & (D / 16 - 1)) << 4);
}

// C consecutive columns of this thread's lane, not waited for.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  static_assert(C == 4 || C == 8 || C == 16, "4, 8 or 16 columns");
  if constexpr (C == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(taddr));
  } else if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
  } else {
    tmem_ld16f(taddr, v);
  }
}

// Wait for the loads above; no use of the values is scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// Values 2 g and 2 g + 1 of an array at a 16-byte boundary, read four at a time.
__device__ __forceinline__ Pair pair_at(const float* x, int g) {
  const float4 v = *reinterpret_cast<const float4*>(x + (g & ~1) * 2);
  return g & 1 ? pair(v.z, v.w) : pair(v.x, v.y);
}

// v = the sum over PARTS parts, part c in columns c * NH ..., of part c / kStep^c.
template <int PARTS, int NH, int NHW>
__device__ __forceinline__ void load_parts(uint32_t taddr, Pair* v) {
  constexpr int kOnce = NHW < 8 ? NHW : 8;  // more would not fit the registers
  const Pair by = pair(1.f / kStep, 1.f / kStep);
#pragma unroll
  for (int first = 0; first < NHW; first += kOnce) {
    float part[PARTS * kOnce];
#pragma unroll
    for (int c = 0; c < PARTS; ++c) tmem_ld<kOnce>(taddr + c * NH + first, part + c * kOnce);
    tmem_wait<PARTS * kOnce>(part);
#pragma unroll
    for (int g = 0; g < kOnce / 2; ++g) {
      Pair x = pair(part[(PARTS - 1) * kOnce + 2 * g], part[(PARTS - 1) * kOnce + 2 * g + 1]);
#pragma unroll
      for (int c = PARTS - 2; c >= 0; --c) {
        const Pair next = pair(part[c * kOnce + 2 * g], part[c * kOnce + 2 * g + 1]);
        x = fma2(x, by, next);
      }
      v[first / 2 + g] = x;
    }
  }
}

// The maximum over a warp's lanes.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Four e5m2 codes of two packed pairs.
__device__ __forceinline__ uint32_t e5m2x4(uint32_t lo, uint32_t hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 a, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 b, %2;\n\tmov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "r"(lo), "r"(hi));
  return r;
}

// kStep (h - the lower or upper two codes): exact (a code is the upper byte of its
// fp16 value).
template <int UPPER>
__device__ __forceinline__ uint32_t remainder_of(uint32_t h2, uint32_t codes) {
  const uint32_t back = __byte_perm(codes, 0u, UPPER ? 0x3424 : 0x1404);
  const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h2),
                                    *reinterpret_cast<const __half2*>(&back)),
                            __float2half2_rn(kStep));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// One work item: up to NH rows of sequence s and one KV head over the partition
// [t_begin, t_end) of the context (no tiles: nothing to do).
struct alignas(16) Item {
  int s, kvh, part, row_first, rows;  // rows [row_first, + rows) of the sequence's
  int query0, queries;                // its first row of q, and how many
  int ctx, base, t_begin, t_end, n_tiles, nparts_seq, unused[3];
};
static_assert(sizeof(Item) == 64, "four 16-byte words");

// Sequence s's queries (first row, count); counts that do not fit are cut.
__device__ __forceinline__ void item_queries(const AttnFp8Params& p, int s, int ctx, Item* it,
                                             bool* bad) {
  if (p.query_start == nullptr) {
    it->query0 = s;
    it->queries = 1;
    it->base = ctx;
    return;
  }
  const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
  const bool there = q0 >= 0 && q1 >= q0 && q1 <= p.total_queries;
  const int n = there ? min(q1 - q0, p.max_query_len) : 0;
  *bad = !there || n < q1 - q0 || n > ctx;
  it->query0 = there ? q0 : 0;
  it->queries = n;
  it->base = max(ctx - n, 0);
}

template <int NH>
__device__ __forceinline__ Item item_at(const AttnFp8Params& p, int j, bool report) {
  Item it{};
  const int chunk = j % p.chunks;
  int r = j / p.chunks;
  it.kvh = r % p.num_kv_heads;
  r /= p.num_kv_heads;
  it.s = r % p.num_seqs;
  it.part = r / p.num_seqs;  // last: the shorter last partitions fill what is left
  const int raw = __ldg(p.context_lens + it.s);
  const long long cap = min((long long)p.max_context_len,
                            (long long)p.max_blocks_per_seq * p.block_size);
  it.ctx = raw < 0 ? 0 : (raw > cap ? (int)cap : raw);
  bool bad = false;
  item_queries(p, it.s, it.ctx, &it, &bad);
  if (report && (bad || raw != it.ctx) && it.part == 0 && chunk == 0)
    atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
  it.row_first = chunk * NH;
  it.rows = min(NH, it.queries * p.group - it.row_first);
  it.t_begin = it.part * p.partition_size;
  it.t_end = partition_end(it.ctx, it.t_begin, p.partition_size);
  it.n_tiles = it.rows > 0 && it.t_begin < it.t_end ? (it.t_end - it.t_begin + kKeys - 1) / kKeys
                                                    : 0;
  it.nparts_seq = context_partitions(it.ctx, p.partition_size);
  return it;
}

// Output row (query row * Hq + head) of the item's row r.
__device__ __forceinline__ int output_row(const AttnFp8Params& p, const Item& it, int r) {
  const int row = it.row_first + r, j = row / p.group;
  return (it.query0 + j) * p.num_q_heads + it.kvh * p.group + (row - j * p.group);
}

// One arrival for what every lane of the warp has done.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tbar.warp.sync 0xffffffff;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

// mbar_wait_warp that looks at the clock and the status only now and then.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, unsigned int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_ns();
  for (uint32_t asked = 1;; ++asked) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (asked % 64 == 0 &&
        __any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs || timed_out(status))) {
      atomicOr(status, PKV_DEV_WAIT_TIMEOUT);
      return false;
    }
  }
}

// The items a warp goes through, in the order the item warp hands them out.
struct ItemWalk {
  const Item* items;
  uint64_t* full;
  uint64_t* empty;
  unsigned int* status;
  int n = 0;

  // False after the last one, or when the wait gave up (the whole warp agrees).
  __device__ __forceinline__ bool next(Item* it) {
    const int b = n % kItemBufs;
    if (!wait_warp(&full[b], (n / kItemBufs) & 1, status)) return false;
    *it = items[b];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[b]);
    ++n;
    return it->n_tiles > 0;
  }
};

// Ask for the index of a CTA of this grid that has not started, which then
// never does: this CTA works in its place.  The answer comes as 16 bytes.
__device__ __forceinline__ void take_cta(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}
// The index, or -1 where none was left.
__device__ __forceinline__ int taken_cta(const void* answer) {
  const volatile unsigned long long* a = static_cast<const volatile unsigned long long*>(answer);
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\tmov.b128 a, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(ok), "+r"(x)
      : "l"(a[0]), "l"(a[1]));
  return ok ? (int)x : -1;
}

// The sums over a warp's lanes of N values: lane l returns that of value
// l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float* v) {
  const int lane = threadIdx.x & 31;
  int mask = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, mask /= 2) {
    const bool upper = lane & mask;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[n + i] : v[i], send = upper ? v[i] : v[n + i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
  }
  float r = v[0];
  for (; mask >= 1; mask /= 2) r += __shfl_xor_sync(0xffffffffu, r, mask);
  return r;
}

// Entries [0, n) of a row of the block table, a warp's 32 at a time, the next
// 32 on their way.
struct TableWindow {
  const int32_t* row;
  int n, first = 0, now, ahead;

  __device__ __forceinline__ TableWindow(const int32_t* r, int entries) : row(r), n(entries) {
    now = load(0);
    ahead = load(32);
  }
  __device__ __forceinline__ int load(int at) const {
    const int i = at + (threadIdx.x & 31);
    return i < n ? __ldg(row + i) : 0;
  }
  // Lane l's entry i + at(l); i + at(l) never goes back by more than the window.
  __device__ __forceinline__ int entry(int i, int at) {
    if (i >= first + 32) {
      first += 32;
      now = ahead;
      ahead = load(first + 32);
    }
    return __shfl_sync(0xffffffffu, now, (i - first + at) & 31);
  }
};

// True if any of the 128 threads of key warpgroup kg passes true.
__device__ __forceinline__ bool group_any(int kg, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %2, 0;\n\t"
      "bar.red.or.pred po, %1, 128, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(1 + kg), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

// True if any of the threads of the KG key warpgroups passes true.
template <int KG>
__device__ __forceinline__ bool keys_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %3, 0;\n\t"
      "bar.red.or.pred po, %1, %2, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "n"(1 + KG), "n"(128 * KG), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tma_load_run(void* dst, const CUtensorMap* map, int row,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(smem_addr(bar))
      : "memory");
}

// Eight bytes, or zeros where `bytes` is 0.
__device__ __forceinline__ void copy8_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// Sixteen bytes, or zeros where `bytes` is 0.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// The e4m3 parts of a query row that D / 8 neighbouring lanes hold, lane c its
// elements 8 c ..., as row `row` of each part in shared memory; returns the power
// of two that they are to be multiplied with (NaN for a row with a NaN or an
// infinity).
template <typename T, int NH, int D>
__device__ __forceinline__ float split_row(uint4 x, int row, int c, unsigned char* dst) {
  constexpr int kLanes = D / 8;
  uint32_t top = max_magnitude(x);
#pragma unroll
  for (int mk = kLanes / 2; mk >= 1; mk >>= 1)
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, mk));
  top = max(top & 0xffffu, top >> 16);
  const bool finite = top < Magnitude<T>::kInf;
  const int e = row_exponent(finite ? Magnitude<T>::value(top) : 0.f);
  const float inv = finite ? pow2(-e) : 0.f;
  const uint32_t words[4] = {x.x, x.y, x.z, x.w};
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Cvt<T>::to_float2(words[i]);
    y[2 * i] = finite ? f.x * inv : 0.f;
    y[2 * i + 1] = finite ? f.y * inv : 0.f;
  }
#pragma unroll
  for (int part = 0; part < kQParts; ++part) {
    uint32_t codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      codes[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE,
                                          __NV_E4M3);
      const float2 back = decode2(codes[i]);
      y[2 * i] = (y[2 * i] - back.x) * kStep;
      y[2 * i + 1] = (y[2 * i + 1] - back.y) * kStep;
    }
    if (row < NH)
      *reinterpret_cast<uint2*>(dst + swizzled<D>(part * NH + row, c * 8)) =
          make_uint2(codes[0] | codes[1] << 16, codes[2] | codes[3] << 16);
  }
  return finite ? pow2(e) : CUDART_NAN_F;
}

template <typename T, int NH, int D>
__global__ void __launch_bounds__(Shape<NH, D>::kThreads, Shape<NH, D>::kPerSm)
    attn_fp8_kernel(const AttnFp8Params p, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, int num_items, bool takes) {
  using L = Shape<NH, D>;
  constexpr int S = L::kStages, SB = L::SB, PB = kBufs, SC = L::kScaleStages, NHW = L::NHW,
                QB = L::kQBufs;
  grid_dep_wait();
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sK = smem;
  unsigned char* sV = smem + S * L::kTile;
  unsigned char* sQ = smem + L::kQ;
  unsigned char* sP = smem + L::kP;
  uint16_t* sScales = reinterpret_cast<uint16_t*>(smem + L::kScales);
  unsigned long long* sMasks = reinterpret_cast<unsigned long long*>(smem + L::kMasks);
  float* sFactors = reinterpret_cast<float*>(smem + L::kFactors);
  int* sRows = reinterpret_cast<int*>(smem + L::kRows);
  Item* sItems = reinterpret_cast<Item*>(smem + L::kItems);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBar);  // [S] tile landed
  uint64_t* k_empty = k_full + S;   // [S] its MMAs are done (commit)
  uint64_t* v_full = k_empty + S;   // [S]
  uint64_t* v_empty = v_full + S;   // [S]
  uint64_t* s_full = v_empty + S;   // [SB] S^T computed (commit)
  uint64_t* s_free = s_full + SB;   // [SB] read by the key warpgroups
  uint64_t* p_full = s_free + SB;   // [PB] weights written (and O^T of the item before read)
  uint64_t* p_free = p_full + PB;   // [PB] their MMAs are done (commit)
  uint64_t* c_full = p_free + PB;   // [SC] the tile's scales landed
  uint64_t* q_full = c_full + SC;   // [QB] the parts of an item's rows of q written
  uint64_t* q_free = q_full + QB;   // [QB] its S^T computed (commit)
  uint64_t* m_full = q_free + QB;   // [2] its output rows, factors and masks written
  uint64_t* m_free = m_full + 2;    // [2] read
  uint64_t* drain = m_free + 2;     // [2] each issuer's last MMAs finished
  uint64_t* i_full = drain + 2;     // [kItemBufs] item written
  uint64_t* i_free = i_full + kItemBufs;  // [kItemBufs] read by every warp
  uint64_t* ticket = i_free + kItemBufs;  // the answer landed
  uint64_t* q_first = ticket + 1;         // q_full of the first item
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int b = 0; b < SB; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4 * L::KG);  // a lane of each key warp arrives
    }
    for (int b = 0; b < PB; ++b) {
      mbar_init(&p_full[b], 4 * L::KG);
      mbar_init(&p_free[b], 1);
    }
    for (int b = 0; b < SC; ++b) mbar_init(&c_full[b], 32);
    for (int b = 0; b < QB; ++b) {
      mbar_init(&q_full[b], L::kQWarps);
      mbar_init(&q_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m_full[b], L::kQWarps);
      mbar_init(&m_free[b], 4 * L::KG);
      mbar_init(&drain[b], 1);
    }
    for (int b = 0; b < kItemBufs; ++b) {
      mbar_init(&i_full[b], 1);
      mbar_init(&i_free[b], L::kReaders);
    }
    mbar_init(ticket, 1);
    mbar_init(q_first, 4 * L::KG);
    fence_barrier_init();
  }
  if (warp == L::kSWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(L::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ItemWalk walk{sItems, i_full, i_free, p.status};
  Item it;
  // (Said in each branch: where they meet, the compiler counts on the least.)
  auto few_registers = [] {
    if constexpr (L::KG > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(few_regs(L::KG)));
  };

  if (warp > L::kReaders) {
    few_registers();  // the idle warp
  } else if (warp == L::kItemWarp) {
    few_registers();
    // ------------------------------------------------------------ item warp
    // Starts with the CTA's own index and goes on with those of CTAs that have
    // not started, so that an SM whose items are short takes more of them.
    void* answer = smem + L::kTicket;
    int j = blockIdx.x, n = 0, asked = 0;
    bool ok = true;
    while (ok && j >= 0) {
      if (takes && lane == 0) {
        mbar_arrive_expect_tx(ticket, 16);
        take_cta(answer, ticket);
      }
      // (A CTA stands for more than one item where there are very many, most of
      // them past the end of a context.)
      for (int i = j; ok && i < num_items && i >= 0; i += gridDim.x) {
        it = item_at<NH>(p, i, lane == 0);
        if (it.n_tiles > 0) {
          const int b = n % kItemBufs;
          ok = n < kItemBufs || wait_warp(&i_free[b], (n / kItemBufs - 1) & 1, p.status);
          if (ok && lane == 0) {
            sItems[b] = it;
            mbar_arrive(&i_full[b]);
          }
          ++n;
        } else if (it.ctx == 0 && it.part == 0) {  // nothing to see: zeros
          constexpr int kWords = D / 8;
          for (int w = lane; w < it.rows * kWords; w += 32)
            reinterpret_cast<uint4*>(p.out)[(size_t)output_row(p, it, w / kWords) * kWords +
                                            w % kWords] = make_uint4(0, 0, 0, 0);
        }
      }
      if (!takes) break;
      if (!ok || !wait_warp(ticket, asked & 1, p.status)) {
        mbar_drain(ticket, asked & 1);  // the answer lands before the CTA leaves
        ok = false;
        break;
      }
      ++asked;
      j = taken_cta(answer);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }
    const int b = n % kItemBufs;
    if (ok && (n < kItemBufs || wait_warp(&i_free[b], (n / kItemBufs - 1) & 1, p.status)) &&
        lane == 0) {
      sItems[b].n_tiles = 0;  // the end
      mbar_arrive(&i_full[b]);
    }
    __syncwarp();
  } else if (warp == L::kKWarp || warp == L::kVWarp) {
    few_registers();
    // ----------------------------------------------------------- producers
    // Tile i covers keys [t_begin + 128 i, + 128): runs of B rows, one block
    // each, lane l copies run l.  The K warp brings the scales as well: lane l
    // those of keys 4 l .. 4 l + 3 (one block: B >= 8).
    const bool is_k = warp == L::kKWarp;
    const CUtensorMap* map = is_k ? &kmap : &vmap;
    unsigned char* ring = is_k ? sK : sV;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    const int B = p.block_size, shift = 31 - __clz(B), runs = kKeys >> shift;
    prefetch_tensormap(map);
    int kt = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      const int blocks = (it.t_end - it.t_begin + B - 1) >> shift;
      TableWindow table(p.block_tables + (size_t)it.s * p.max_blocks_per_seq +
                            (it.t_begin >> shift), blocks);
      for (int i = 0; i < it.n_tiles; ++i, ++kt) {
        const int st = kt % S;
        const int nseg = min(runs, blocks - i * runs);
        int phys = table.entry(i * runs, lane & 15);
        int phys4 = is_k ? table.entry(i * runs, (lane * 4) >> shift) : 0;
        if ((unsigned)phys >= (unsigned)p.num_blocks) {
          if (lane < nseg) atomicOr(p.status, PKV_DEV_BAD_BLOCK_ID);
          phys = 0;
        }
        if ((unsigned)phys4 >= (unsigned)p.num_blocks) phys4 = 0;
        if (kt >= S && !wait_warp(&empty[st], ((kt / S) - 1) & 1, p.status)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nseg * D) << shift);
        __syncwarp();
        if (lane < nseg)
          tma_load_run(ring + st * L::kTile + ((lane * D) << shift), map,
                       (phys * p.num_kv_heads + it.kvh) << shift, &full[st]);
        if (is_k) {
          const int key = it.t_begin + i * kKeys + lane * 4;
          const size_t row = (((size_t)phys4 * p.num_kv_heads + it.kvh) << shift) + (key & (B - 1));
          const int bytes = key < it.t_end ? 8 : 0;
          uint16_t* to = sScales + 2 * (kt % SC) * kKeys + lane * 4;
          copy8_async(to, p.k_scales + (bytes ? row : 0), bytes);
          copy8_async(to + kKeys, p.v_scales + (bytes ? row : 0), bytes);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_addr(&c_full[kt % SC]))
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // After a timeout, copies still in flight land before the CTA leaves.
    if (timed_out(p.status))
      for (int i = kt > S ? kt - S : 0; i < kt; ++i) mbar_drain(&full[i % S], (i / S) & 1);
    __syncwarp();
  } else if (warp >= L::kQWarp) {
    few_registers();
    // -------------------------------------------------------------- Q warps
    // Warp w brings its rows into shared memory as they are, then splits them:
    // a row lies in D / 8 lanes.  Rows past the item's are zeros.  With many rows
    // the first item, which nothing hides, is split by all the key warps (8
    // sequences with trees of 64 over groups of three 64 -> 60 us).
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kMine = NH / L::kQWarps,
                  kRound = L::kRawRows / L::kQWarps;
    const int w = warp - L::kQWarp, c = lane % kLanes;
    unsigned char* raw = smem + L::kQRaw + w * kRound * D * 2;
    while (walk.next(&it)) {
      const int k_item = walk.n - 1, b = k_item % QB, mb = k_item & 1;
      if (L::kKeysSplit && k_item == 0) continue;  // the key warps' own
      const int my_row = w * kMine + lane;  // lane l knows the warp's row l
      const int my_out = output_row(p, it, min(my_row, it.rows - 1));
      unsigned long long mask = 0;
      if (p.tree_masks)
        mask = (unsigned long long)__ldg(reinterpret_cast<const long long*>(p.tree_masks) +
                                         my_out / p.num_q_heads);
      bool ok = true;
      unsigned char* dst = sQ + b * L::kQBytes;
#pragma unroll 1
      for (int first = 0; first < kMine; first += kRound) {
#pragma unroll 1
        for (int r = lane / kLanes; r < kRound; r += kAtOnce) {
          const int row = w * kMine + first + r;
          const int from = __shfl_sync(0xffffffffu, my_out, first + r);
          copy16_async(raw + (r * kLanes + c) * 16,
                       static_cast<const T*>(p.q) + (size_t)from * D + c * 8,
                       row < it.rows ? 16 : 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (first == 0) {
          ok = (k_item < QB || wait_warp(&q_free[b], (k_item / QB - 1) & 1, p.status)) &&
               (k_item < 2 || wait_warp(&m_free[mb], (k_item / 2 - 1) & 1, p.status));
          if (!ok) break;
        }
#pragma unroll 1
        for (int r = lane / kLanes; r < kRound; r += kAtOnce) {
          const uint4 x = *reinterpret_cast<const uint4*>(raw + (r * kLanes + c) * 16);
          const int row = w * kMine + first + r;
          const float factor = split_row<T, NH, D>(x, row, c, dst);
          if (c == 0) sFactors[mb * NH + row] = p.qscale * factor;
        }
      }
      if (!ok) break;
      if (lane < kMine) {
        sRows[mb * NH + my_row] = my_out;
        sMasks[mb * NH + my_row] = mask;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      arrive_warp(&q_full[b]);
      arrive_warp(&m_full[mb]);
    }
    __syncwarp();
  } else if (warp == L::kSWarp || warp == L::kOWarp) {
    few_registers();
    // ------------------------------------------------------------ issuers
    const bool is_s = warp == L::kSWarp;
    const uint32_t idesc = is_s ? instr(false, L::NS, kKeys) : instr(true, L::NO, D);
    const uint32_t aK = smem_addr(sK), aV = smem_addr(sV), aQ = smem_addr(sQ),
                   aP = smem_addr(sP);
    int kt = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (is_s) {
        const int k_item = walk.n - 1, b = k_item % QB;
        const bool own = L::kKeysSplit && k_item == 0;
        const int filled = own ? 0 : k_item / QB - (L::kKeysSplit && b == 0);
        if (!wait_warp(own ? q_first : &q_full[b], filled & 1, p.status)) break;
        for (int i = 0; i < it.n_tiles; ++i, ++kt) {
          const int st = kt % S;
          if (!wait_warp(&k_full[st], (kt / S) & 1, p.status) ||
              (kt >= SB && !wait_warp(&s_free[kt % SB], ((kt / SB) - 1) & 1, p.status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          // 32 dimensions per MMA: a 32-byte step inside the swizzled rows.
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma_f8_warp(tmem + (kt % SB) * L::NS,
                        desc(aK + st * L::kTile + ks * 32, 16, 8 * D, L::kSwizzle),
                        desc(aQ + b * L::kQBytes + ks * 32, 16, 8 * D, L::kSwizzle), idesc,
                        ks > 0 ? 1u : 0u);
          mma_commit_warp(&s_full[kt % SB]);
          mma_commit_warp(&k_empty[st]);
        }
        if (ok) mma_commit_warp(&q_free[b]);
      } else {
        for (int i = 0; i < it.n_tiles; ++i, ++kt) {
          const int st = kt % S;
          if (!wait_warp(&v_full[st], (kt / S) & 1, p.status) ||
              !wait_warp(&p_full[kt % PB], (kt / PB) & 1, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // 32 keys per MMA, four groups of 8.  V: the D columns are one
          // swizzled atom, groups 8 D bytes apart.  P: 16-byte columns 128
          // bytes apart, groups 8 NO bytes apart.
#pragma unroll
          for (int ks = 0; ks < kKeys / 32; ++ks)
            mma_f8_warp(tmem + L::kColO,
                        desc(aV + st * L::kTile + ks * 32 * D, 16, 8 * D, L::kSwizzle),
                        desc(aP + (kt % PB) * L::kPBuf + ks * 32 * L::NO, 8 * L::NO, 128, 0),
                        idesc, (i > 0 || ks > 0) ? 1u : 0u);
          mma_commit_warp(&p_free[kt % PB]);
          mma_commit_warp(&v_empty[st]);
        }
      }
    }
    uint64_t* d = &drain[is_s ? 0 : 1];
    mma_commit_warp(d);
    mbar_drain(d, 0);
    __syncwarp();
  } else {
    if constexpr (L::KG > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kKeyRegs));
    // ----------------------------------------------------- key warpgroups
    // Code that runs once per item or seldom is kept short (loops that stay
    // loops): straight-line code met for the first time runs at the latency of
    // its fetch.
    const int kg = warp >> 2;
    const int t = threadIdx.x & 127;  // key of the tile == tensor-memory lane
    const int hb = kg * NHW;          // first row of this warpgroup
    const int row = lane & (NHW - 1); // the row whose reference this lane keeps
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // the dimension whose outputs this lane holds (D = 64: half of the lanes)
    const int d = D == 128 ? t : (warp & 3) * 16 + lane;
    const bool has_d = D == 128 || lane < 16;
    const int at = (kg * 4 + (warp & 3)) * NHW;
    float* tops = reinterpret_cast<float*>(smem + L::kTop) + kg * 4 * NHW;
    float* sums = reinterpret_cast<float*>(smem + L::kSum) + kg * 4 * NHW;
    float* refs = reinterpret_cast<float*>(smem + L::kRef) + at;      // minus the references
    int* marks = reinterpret_cast<int*>(smem + L::kMarks) + kg * 4;
    float* alphas = reinterpret_cast<float*>(smem + L::kAlpha) + at;  // (this warp's copies)
    float* shifts = reinterpret_cast<float*>(smem + L::kShift) + at;
    int kt = 0, sc = 0;
    uint32_t sc_phase = 0;
    bool ok = true;
    for (;;) {
      const bool more = walk.next(&it);
      if (keys_any<L::KG>(!more)) break;  // the key warps leave together
      const int k_item = walk.n - 1, mb = k_item & 1;
      if (L::kKeysSplit && k_item == 0) {
        // Each key warp splits its share of the rows, one or two at a time.
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kShare = NHW / 4;
        const int c = lane % kLanes;
#pragma unroll 1
        for (int r = lane / kLanes; r - lane / kLanes < kShare; r += kAtOnce) {
          const int q_row = r < kShare ? warp * kShare + r : NH;
          const bool there = q_row < it.rows;
          const int from = output_row(p, it, min(q_row, it.rows - 1));
          uint4 x = make_uint4(0, 0, 0, 0);
          if (there)
            x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                     (size_t)from * D) + c);
          if (c == 0 && q_row < NH) {
            sRows[q_row] = from;
            if (p.tree_masks)
              sMasks[q_row] = (unsigned long long)__ldg(
                  reinterpret_cast<const long long*>(p.tree_masks) + from / p.num_q_heads);
          }
          const float factor = split_row<T, NH, D>(x, q_row, c, sQ);
          if (c == 0 && q_row < NH) sFactors[q_row] = p.qscale * factor;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        arrive_warp(q_first);
        ok = ok && mbar_wait(q_first, 0, p.status);
      } else {
        // (Not q_full, which may be filled again before the last key warp looks.)
        ok = ok && mbar_wait(&m_full[mb], (k_item / 2 - (L::kKeysSplit && mb == 0)) & 1, p.status);
      }
      const float* factors = sFactors + mb * NH + hb;
      if (L::KG > 1 && hb >= it.rows) {
        // None of this warpgroup's rows is there: it only hands the buffers on.
        // (What they hold for its rows comes to nothing that is stored.)
        for (int i = 0; i < it.n_tiles; ++i, ++kt) {
          const int sb = kt % SB, pb = kt % PB;
          ok = ok && mbar_wait(&s_full[sb], (kt / SB) & 1, p.status);
          arrive_warp(&s_free[sb]);
          if (p.tree_masks != nullptr && min(it.t_begin + (i + 1) * kKeys, it.t_end) > it.base)
            named_barrier_sync(1 + L::KG, 128 * L::KG);
          if (kt >= PB) ok = ok && mbar_wait(&p_free[pb], ((kt / PB) & 1) ^ 1, p.status);
          arrive_warp(&p_full[pb]);
        }
        sc = kt % SC;
        sc_phase = (kt / SC) & 1;
        arrive_warp(&m_free[mb]);
        continue;
      }
      // Rows past the item's get weights of zero by their reference.
      float nm = hb + row < it.rows ? 0.f : -CUDART_INF_F;
      bool unset = hb + row < it.rows;  // nm is of no weight yet
      if (lane < NHW) refs[row] = nm;
      __syncwarp();
      Pair l_part[NHW / 2];
#pragma unroll
      for (int g = 0; g < NHW / 2; ++g) l_part[g] = pair(0.f, 0.f);
      int ref_v = kNoScale;  // E
      bool far = false;      // rows were added apart
      for (int i = 0; i < it.n_tiles; ++i, ++kt) {
        const int key0 = it.t_begin + i * kKeys;
        const int nvalid = min(kKeys, it.t_end - key0);
        const bool valid = t < nvalid;
        const int sb = kt % SB;
        const uint32_t s_phase = (kt / SB) & 1, p_phase = (kt / PB) & 1;
        const int pb = kt % PB;
        // A wait that gives up (never expected) leaves ok false; the loop runs
        // on without waiting, so that every named barrier stays matched, and
        // nothing it computes is stored.
        // (Both are asked before either answer is looked at.)
        const bool c_here = mbar_try_wait(&c_full[sc], sc_phase);
        const bool s_here = mbar_try_wait(&s_full[sb], s_phase);
        if (!(c_here && s_here))
          ok = ok && mbar_wait(&c_full[sc], sc_phase, p.status) &&
               mbar_wait(&s_full[sb], s_phase, p.status);
        __syncwarp();
        tc_fence_after();
        const uint16_t* scales = sScales + 2 * sc * kKeys + t;
        if (++sc == SC) {
          sc = 0;
          sc_phase ^= 1;
        }
        const float ks = scale_value(scales[0]);
        uint32_t vb = scales[kKeys];
        if (i == 0) {
          // E: the tile's largest scale, looked for by every warp (with a NaN in it, or
          // drafts that may not count, looked at again below).
          uint2 four = *reinterpret_cast<const uint2*>(scales - t + kKeys + lane * 4);
          const int n = nvalid - lane * 4;  // of the four, in the context
          four.x &= (n > 1 ? 0xffffff80u : n > 0 ? 0xff80u : 0u);
          four.y &= (n > 3 ? 0xffffff80u : n > 2 ? 0xff80u : 0u);
          const uint32_t two = __vmaxu2(four.x, four.y);
          const int most = (int)__reduce_max_sync(0xffffffffu, max(two & 0xff80u, two >> 16));
          if (most >= 0x80 && most < 0x7f80) ref_v = reference_of(most);
        }
        Pair y[NHW / 2];
        load_parts<kQParts, NH, NHW>(tmem + sb * L::NS + hb + lane_base, y);
        tc_fence_before();
        arrive_warp(&s_free[sb]);

        uint32_t seen = valid ? 0xffffffffu : 0u;
        const bool tail = p.tree_masks != nullptr && key0 + nvalid > it.base;
        const int st = kt % S;
        if (tail) {
          // Drafted positions: a row sees those of its mask.  What is masked
          // must not reach the second product, whose zero weights do not hide
          // a NaN code: such a row of V counts as NaN by its scale, and its
          // codes are cleared below.
          const int rel = key0 + t - it.base;
          if (valid && rel >= 0) {
            const unsigned long long* masks = sMasks + mb * NH + hb;
            uint32_t bits = 0;
#pragma unroll 4
            for (int g = 0; g < NHW; ++g) bits |= (uint32_t)((masks[g] >> rel) & 1) << g;
            seen = bits;
          }
          ok = ok && mbar_wait(&v_full[st], (kt / S) & 1, p.status);
          bool nan = false;
          uint4* v_row = reinterpret_cast<uint4*>(sV + st * L::kTile + t * D);
          if (valid && rel >= 0) {
#pragma unroll 2
            for (int c = 0; c < D / 16; ++c) {
              const uint4 w = v_row[(c + t) % (D / 16)];  // (neighbours in different banks)
              nan |= (__vcmpeq4(w.x & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                      __vcmpeq4(w.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                      __vcmpeq4(w.z & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                      __vcmpeq4(w.w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0;
            }
          }
          if constexpr (L::KG > 1) named_barrier_sync(1 + L::KG, 128 * L::KG);  // both have read
          if (nan) {
            vb = kNanScale;
            if (kg == 0)
#pragma unroll 2
              for (int c = 0; c < D / 16; ++c) v_row[c] = make_uint4(0, 0, 0, 0);
          }
        }
        // What this key's V scale does: y = x + lv, l gets p * 2^-lv.  Scales out of
        // the band, NaN among them, are looked after below.
        vb &= 0xff80u;
        if (nvalid < kKeys && !valid) vb = ref_v + kBelow * 128;
        const uint32_t in_band = vb - ref_v;
        const bool odd = in_band > kBand;
        const float lvf = fmaf(__uint_as_float(0x4b000000u + in_band), 1.f / 128,  // 2^23 + in_band
                               -(65536.f + kBelow));
        int lv_bits = in_band;  // (lv + kBelow) * 128
        const Pair ks2 = pair(ks, ks), lv2 = pair(lvf, lvf);
#pragma unroll
        for (int g = 0; g < NHW / 2; ++g) y[g] = fma2(y[g], mul2(pair_at(factors, g), ks2), lv2);
        if (tail || nvalid < kKeys) {
#pragma unroll
          for (int g = 0; g < NHW / 2; ++g) {
            const float2 v = both(y[g]);
            y[g] = pair(seen >> (2 * g) & 1 ? v.x : -CUDART_INF_F,
                        seen >> (2 * g + 1) & 1 ? v.y : -CUDART_INF_F);
          }
        }
        float2 e[NHW / 2];  // y - m, then the weights
        float top = -CUDART_INF_F;
#pragma unroll
        for (int g = 0; g < NHW / 2; ++g) {
          e[g] = both(add2(y[g], pair_at(refs, g)));
          top = fmax3(top, e[g].x, e[g].y);
        }
        if (group_any(kg, top > kExceed || unset || odd)) {
          bool low = false, apart = false;  // this key, some of the tile's are added apart
          float shrink = 1.f;
          const bool again = i == 0 && tail;
          if (__builtin_expect(group_any(kg, odd || again), 0)) {
            const bool v_nan = vb >= 0x7f80u;
            const int of_warp =
                __reduce_max_sync(0xffffffffu, seen != 0 && !v_nan ? (int)vb : 0);
            if (lane == 0) marks[warp & 3] = of_warp;
            named_barrier_sync(1 + kg, 128);
            const int largest = max(max(marks[0], marks[1]), max(marks[2], marks[3]));
            if (again) ref_v = kNoScale;  // (it may be of drafts that no row sees)
            if (largest >= 0x80 && (ref_v == kNoScale || largest > ref_v + kBand)) {
              // E moves, and the O^T so far with it (below).
              const int old = ref_v;
              ref_v = reference_of(largest);
              if (i > 0) shrink = old == kNoScale || ref_v - old > 126 * 128 ? 0.f : pow2((old - ref_v) / 128);
            }
            const int at = (int)vb - ref_v;
            const int lv = min(max(at >> 7, 0), kAbove + kBelow) - kBelow;
            const float by = v_nan ? CUDART_NAN_F : (float)lv - lvf;
            lv_bits = (lv + kBelow) * 128;
#pragma unroll
            for (int g = 0; g < NHW / 2; ++g) {  // (-infinity: not seen)
              if (e[g].x > -CUDART_INF_F) e[g].x += by;
              if (e[g].y > -CUDART_INF_F) e[g].y += by;
            }
            low = seen != 0 && !v_nan && at < 0;
            apart = group_any(kg, low);
          }
          // The tile's maxima per row, then the rows whose reference moves:
          // lane r of each warp settles row r.
          float mine = 0.f;
#pragma unroll
          for (int g = 0; g < NHW / 2; ++g) {
            const float a = warp_max(e[g].x), b = warp_max(e[g].y);
            if (row / 2 == g) mine = row & 1 ? b : a;
          }
          if (lane < NHW) tops[(warp & 3) * NHW + row] = mine;
          named_barrier_sync(1 + kg, 128);
          const float mt = fmax3(fmaxf(tops[row], tops[NHW + row]), tops[2 * NHW + row],
                                 tops[3 * NHW + row]);
          // (All that have grown, now that some must.)
          const bool moves = mt > (unset ? -CUDART_INF_F : kPlace);
          const float shift = moves ? kPlace - mt : 0.f;
          nm += shift;
          if (lane < NHW) {
            refs[row] = nm;
            shifts[row] = shift;
            alphas[row] = unset ? 0.f : ex2(shift);  // (an unset row has no weights yet)
          }
          unset = unset && mt == -CUDART_INF_F;
          const bool moved = __any_sync(0xffffffffu, moves);  // (orders the stores, too)
          __syncwarp();
#pragma unroll
          for (int g = 0; g < NHW / 2; ++g) {
            l_part[g] = mul2(l_part[g], pair_at(alphas, g));
            e[g] = both(add2(pair(e[g].x, e[g].y), pair_at(shifts, g)));
          }
          if (__builtin_expect(shrink != 1.f, 0)) {
            if (lane < NHW) alphas[row] *= shrink;
            __syncwarp();
          }
          if (i > 0 && (moved || shrink != 1.f)) {
            // O^T holds this item's tiles so far: rescaled once their MMAs are
            // done (P buffer of the previous tile released).
            ok = ok && mbar_wait(&p_free[(kt - 1) % PB], ((kt - 1) / PB) & 1, p.status);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < (far ? kParts + 1 : kParts); ++c) {
              const uint32_t addr =
                  tmem + L::kColO + (c < kParts ? c * NH : L::NO) + hb + lane_base;
              float o[NHW];
              tmem_load_small<NHW>(addr, o);
#pragma unroll
              for (int g = 0; g < NHW; ++g) o[g] *= alphas[g];
              tmem_store_small<NHW>(addr, o);
            }
            tc_fence_before();
          }
          if (__builtin_expect(apart, 0)) {
            // Four keys at a time, the next of each warp: its weights into `tops`,
            // then every thread adds its dimension of the four rows.  Rows of zeros
            // are left out.  The sums get these weights here, the product none.
            ok = ok && mbar_wait(&v_full[st], (kt / S) & 1, p.status);
            named_barrier_sync(1 + kg, 128);  // the maxima have been read
            const unsigned char* v_tile = sV + st * L::kTile;
            uint32_t some = 0;
            if (low && vb >= 0x80u) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                const uint4 w = reinterpret_cast<const uint4*>(v_tile + t * D)[(c + t) % (D / 16)];
                some |= (w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
              }
            }
            const int down = ((int)vb - ref_v) / 128;  // (below 0 where it is used)
            const float v_rel = down < -126 ? 0.f : pow2(min(down, 0));
            uint32_t todo = __ballot_sync(0xffffffffu, some != 0);
#pragma unroll 1
            for (;;) {
              const int src = __ffs(todo) - 1;
              if (lane == max(src, 0)) {
                marks[warp & 3] = src < 0 ? -1 : t;
                float* to = tops + (warp & 3) * NHW;
#pragma unroll
                for (int g = 0; g < NHW / 2; ++g) {
                  to[2 * g] = ex2(e[g].x) * v_rel;
                  to[2 * g + 1] = ex2(e[g].y) * v_rel;
                }
              }
              __syncwarp();
              if (!group_any(kg, src >= 0)) break;
              float code[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int key = marks[w];
                code[w] = key < 0 || !has_d ? 0.f : decode2(v_tile[swizzled<D>(key, d)]).x;
              }
#pragma unroll 1
              for (int g = 0; g < NHW; g += 4) {
                const uint32_t addr = tmem + L::kColFar + hb + g + lane_base;
                float o[4] = {0.f, 0.f, 0.f, 0.f};
                if (far) tmem_load_small<4>(addr, o);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  if (marks[w] < 0) continue;  // (its weights are none)
                  const float4 x = *reinterpret_cast<const float4*>(tops + w * NHW + g);
                  o[0] = fmaf(x.x, code[w], o[0]);
                  o[1] = fmaf(x.y, code[w], o[1]);
                  o[2] = fmaf(x.z, code[w], o[2]);
                  o[3] = fmaf(x.w, code[w], o[3]);
                }
                tmem_store_small<4>(addr, o);
              }
              far = true;
              todo &= todo - 1;
              named_barrier_sync(1 + kg, 128);  // read, before the next are written
            }
            if (low) {
#pragma unroll
              for (int g = 0; g < NHW / 2; ++g) {  // (lv = -kBelow)
                l_part[g] = fma2(pair(ex2(e[g].x), ex2(e[g].y)),
                                 pair(pow2(kBelow), pow2(kBelow)), l_part[g]);
                e[g] = make_float2(-CUDART_INF_F, -CUDART_INF_F);
              }
            }
            __syncwarp();
          }
        }
        // The weights of this key: rounded to fp16, then split in three.  The
        // buffer was last read by the MMAs of tile kt - PB.
        // (Nothing to wait for in the first PB: their phase before the first counts
        // as completed.)
        const bool p_here = mbar_test_wait(&p_free[pb], p_phase ^ 1);
        const float inv_v = __uint_as_float(((127u + kBelow) << 23) - ((uint32_t)lv_bits << 16));
        const Pair inv2 = pair(inv_v, inv_v);
        uint32_t h[NHW / 2];
#pragma unroll
        for (int g = 0; g < NHW / 2; ++g) {
          e[g] = make_float2(ex2(e[g].x), ex2(e[g].y));
          l_part[g] = fma2(pair(e[g].x, e[g].y), inv2, l_part[g]);
          h[g] = Cvt<__half>::from_float2(e[g].x, e[g].y);
        }
        uint32_t part[kParts][NHW / 4];
#pragma unroll
        for (int g = 0; g < NHW / 4; ++g) {
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            part[c][g] = e5m2x4(h[2 * g], h[2 * g + 1]);
            if (c + 1 < kParts) {
              h[2 * g] = remainder_of<0>(h[2 * g], part[c][g]);
              h[2 * g + 1] = remainder_of<1>(h[2 * g + 1], part[c][g]);
            }
          }
        }
        if (!p_here) ok = ok && mbar_wait(&p_free[pb], p_phase ^ 1, p.status);
        uint4* to = reinterpret_cast<uint4*>(sP + pb * L::kPBuf + (t >> 3) * 8 * L::NO +
                                             (t & 7) * 16);
        if constexpr (NH == 4) {
          to[0] = make_uint4(part[0][0], part[1][0], part[2][0], 0u);
        } else if constexpr (NH == 8) {
          to[0] = make_uint4(part[0][0], part[0][1], part[1][0], part[1][1]);
          to[8] = make_uint4(part[2][0], part[2][1], 0u, 0u);
        } else {
#pragma unroll
          for (int c = 0; c < kParts; ++c)
            to[8 * ((c * NH + hb) / 16)] =
                make_uint4(part[c][0], part[c][1], part[c][2], part[c][3]);
        }
        if (nvalid < kKeys && kg == 0) {
          // The item's last tile: V rows past the context must not feed stale
          // or NaN values into O^T (their weights are 0, but 0 * NaN is NaN).
          ok = ok && mbar_wait(&v_full[st], (kt / S) & 1, p.status);
          if (!valid) {
#pragma unroll 2
            for (int c = 0; c < D / 16; ++c)
              reinterpret_cast<uint4*>(sV + st * L::kTile + t * D)[(c + t) % (D / 16)] =
                  make_uint4(0, 0, 0, 0);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        arrive_warp(&p_full[pb]);
      }

      // Row sums over the 128 keys.
      float l_mine[NHW];
#pragma unroll
      for (int g = 0; g < NHW / 2; ++g) {
        const float2 v = both(l_part[g]);
        l_mine[2 * g] = v.x;
        l_mine[2 * g + 1] = v.y;
      }
      __syncwarp();
      const float sum = warp_sums<NHW>(l_mine);
      if (lane % (32 / NHW) == 0) sums[(warp & 3) * NHW + lane / (32 / NHW)] = sum;
      named_barrier_sync(1 + kg, 128);
      const int last = kt - 1;
      ok = ok && mbar_wait(&p_free[last % PB], (last / PB) & 1, p.status);
      __syncwarp();
      tc_fence_after();
      const int* rows = sRows + mb * NH + hb;
      const int there = it.rows - hb;  // of this warpgroup's rows
      const float l = (sums[row] + sums[NHW + row]) + (sums[2 * NHW + row] + sums[3 * NHW + row]);
      if (lane < NHW) alphas[row] = l == 0.f ? 0.f : __fdividef(1.f, l);
      __syncwarp();
      constexpr int kOut = NHW < 8 ? NHW : 8;
      // 2^E
      const float v_scale = ref_v == kNoScale ? 1.f : pow2((ref_v >> 7) - 127 + kBelow);
      if (__builtin_expect(far, 0)) {  // the rows added apart, into the first part
#pragma unroll 1
        for (int g = 0; g < NHW; g += 4) {
          const uint32_t addr = tmem + L::kColO + hb + g + lane_base;
          float o[4], x[4];
          tmem_load_small<4>(addr, o);
          tmem_load_small<4>(addr + L::NO, x);
#pragma unroll
          for (int u = 0; u < 4; ++u) o[u] += x[u];
          tmem_store_small<4>(addr, o);
        }
      }
#pragma unroll 1
      for (int g = 0; g < NHW && g < there; g += kOut) {
        Pair o[kOut / 2];
        load_parts<kParts, NH, kOut>(tmem + L::kColO + hb + g + lane_base, o);
#pragma unroll
        for (int u = 0; u < kOut; ++u) {
          const float2 v = both(o[u / 2]);
          const float inv = alphas[g + u],
                      x = inv == 0.f ? 0.f : (u & 1 ? v.y : v.x) * inv * v_scale;
          if (!ok || !has_d || g + u >= there) continue;
          if (it.nparts_seq == 1)
            static_cast<T*>(p.out)[(size_t)rows[g + u] * D + d] = static_cast<T>(x);
          else
            p.ws_o[((size_t)rows[g + u] * p.num_parts + it.part) * D + d] = x;
        }
      }
      tc_fence_before();
      if (ok && it.nparts_seq > 1 && t < NHW && t < there) {
        const size_t r = (size_t)rows[t] * p.num_parts + it.part;
        p.ws_m[r] = l == 0.f ? kNoRef : -nm;
        p.ws_l[r] = l;
      }
      arrive_warp(&m_free[mb]);  // the item's rows are read
    }
    grid_dep_launch_dependents();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == L::kSWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(L::kTmemCols));
  }
}

// Merge the partitions of sequences whose context spans more than one:
// out = sum_i w_i o_i / sum_i w_i with w_i = l_i 2^(m_i - max m).  A warp per
// output row.
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_fp8_reduce_kernel(const AttnFp8Params p) {
  constexpr int E = D / 32;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)p.total_queries * p.num_q_heads) return;
  const int query = (int)(row / p.num_q_heads);
  const float* mrow = p.ws_m + row * p.num_parts;
  const float* lrow = p.ws_l + row * p.num_parts;
  const float* orow = p.ws_o + row * p.num_parts * D + lane * E;
  // On their way while the sequence is looked for (a call that splits has two
  // partitions at least); of partitions that are none they are not used.
  auto load = [&](int i, float2* o) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
      o[e] = __ldcg(reinterpret_cast<const float2*>(orow + (size_t)i * D) + e);
  };
  float2 early[2][E / 2];
  load(0, early[0]);
  load(1, early[1]);
  float m0 = -CUDART_INF_F, l0 = 0.f;
  if (lane < p.num_parts) {
    m0 = __ldcg(mrow + lane);
    l0 = __ldcg(lrow + lane);
  }
  int s = query;
  if (p.query_start) {  // the last sequence that starts at or before the query
    int lo = 0, n = p.num_seqs;
    while (n > 1) {  // 32 of the candidates at a time
      const int step = (n + 31) / 32;
      const int i = lo + lane * step;
      const bool before = lane * step < n && __ldg(p.query_start + i) <= query;
      const int k = max(31 - __clz(__ballot_sync(0xffffffffu, before)), 0);
      lo += k * step;
      n = min(step, n - k * step);
    }
    s = lo;
  }
  const int raw = __ldg(p.context_lens + s);
  const long long cap = min((long long)p.max_context_len,
                            (long long)p.max_blocks_per_seq * p.block_size);
  const int ctx = raw < 0 ? 0 : (raw > cap ? (int)cap : raw);
  Item it;
  bool bad;
  item_queries(p, s, ctx, &it, &bad);
  if (query < it.query0 || query >= it.query0 + it.queries) return;
  const int np = context_partitions(ctx, p.partition_size);
  if (np <= 1) return;  // written by the attention kernel
  float M = lane < np ? m0 : -CUDART_INF_F;
  for (int i = lane + 32; i < np; i += 32) M = fmaxf(M, __ldcg(mrow + i));
  M = warp_max(M);
  auto weight = [&](int i) {
    if (i >= np) return 0.f;
    const float l = i < 32 ? l0 : __ldcg(lrow + i), m = i < 32 ? m0 : __ldcg(mrow + i);
    return l == 0.f ? 0.f : l * exp2f(m - M);
  };
  // (The sum first: a weight of more than 1 times an output may pass the range.)
  float sum = 0.f;
  for (int i = lane; i < np; i += 32) sum += weight(i);
#pragma unroll
  for (int mk = 16; mk >= 1; mk >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mk);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int base = 0; base < np; base += 32) {
    const float mine = weight(base + lane) * inv;
    const int n = min(32, np - base);
    auto add = [&](int k, const float2* o) {
      const float w = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        acc[2 * e] = fmaf(w, o[e].x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(w, o[e].y, acc[2 * e + 1]);
      }
    };
    if (base == 0) {
      add(0, early[0]);
      add(1, early[1]);
    }
#pragma unroll 4
    for (int k = base == 0 ? 2 : 0; k < n; ++k) {
      float2 o[E / 2];
      load(base + k, o);
      add(k, o);
    }
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = Cvt<T>::from_float2(acc[2 * e], acc[2 * e + 1]);
}

// The cache's rows of D codes: boxes of a block's rows of one head, D-byte
// swizzle.
bool make_codes_map(CUtensorMap* map, const void* base, long long rows, int head_dim,
                    int block_size) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)head_dim};
  const cuuint32_t box[2] = {(cuuint32_t)head_dim, (cuuint32_t)block_size};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int NH, int D>
cudaError_t launch_shape(const AttnFp8Params& p, const CUtensorMap& km, const CUtensorMap& vm,
                         cudaStream_t stream) {
  using L = Shape<NH, D>;
  static unsigned long long configured = 0;  // bit per device ordinal (< 64)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    err = cudaFuncSetAttribute(attn_fp8_kernel<T, NH, D>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (err != cudaSuccess) return err;
    if constexpr (L::KG > 1) {  // the warpgroups' shares come out of what the launch gives
      cudaFuncAttributes attr;
      err = cudaFuncGetAttributes(&attr, attn_fp8_kernel<T, NH, D>);
      if (err != cudaSuccess) return err;
      if (attr.numRegs < few_regs(L::KG) ||
          (attr.numRegs + 7) / 8 * 8 * L::kThreads <
              128 * L::KG * kKeyRegs + (L::kThreads - 128 * L::KG) * few_regs(L::KG))
        return cudaErrorInvalidConfiguration;
    }
    if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELEASE);
  }
  const int items = p.num_seqs * p.num_kv_heads * p.num_parts * p.chunks;
  const int ctas = std::min(items, kMostCtas);
  // Where the device holds all CTAs at once, none takes over another's: the first to
  // run would take those that are about to start, and leave their SMs idle.
  const bool takes = ctas > p.sms * L::kPerSm;
  err = launch_overlapped(attn_fp8_kernel<T, NH, D>, dim3(ctas), dim3(L::kThreads), L::kBytes,
                          stream, p, km, vm, items, takes);
  if (err != cudaSuccess || p.num_parts <= 1) return err;
  const long long rows = (long long)p.total_queries * p.num_q_heads;
  return launch_overlapped(attn_fp8_reduce_kernel<T, D>, dim3((unsigned)((rows + 3) / 4)),
                           dim3(128), 0, stream, p);
}

template <typename T, int D>
cudaError_t launch_rows(const AttnFp8Params& p, const CUtensorMap& km, const CUtensorMap& vm,
                        cudaStream_t stream) {
  static_assert(kFp8Rows == 64, "the instantiations cover items of up to 64 rows");
  const int rows = p.max_query_len * p.group;
  if (rows <= 4) return launch_shape<T, 4, D>(p, km, vm, stream);
  if (rows <= 8) return launch_shape<T, 8, D>(p, km, vm, stream);
  if (rows <= 16) return launch_shape<T, 16, D>(p, km, vm, stream);
  if (rows <= 32) return launch_shape<T, 32, D>(p, km, vm, stream);
  return launch_shape<T, 64, D>(p, km, vm, stream);
}

}  // namespace

cudaError_t launch_attn_fp8(const AttnFp8Params& p, int head_dim, int dtype, cudaStream_t stream,
                            bool* unsupported) {
  CUtensorMap km, vm;
  const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
  *unsupported = !make_codes_map(&km, p.k_cache, rows, head_dim, p.block_size) ||
                 !make_codes_map(&vm, p.v_cache, rows, head_dim, p.block_size);
  if (*unsupported) return cudaErrorInvalidValue;
  if (dtype == PKV_F16)
    return head_dim == 64 ? launch_rows<__half, 64>(p, km, vm, stream)
                          : launch_rows<__half, 128>(p, km, vm, stream);
  return head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, km, vm, stream)
                        : launch_rows<__nv_bfloat16, 128>(p, km, vm, stream);
}

}  // namespace pkv
