// The C ABI: argument checks, launch planning, and the device status word.
// Nothing here allocates device memory.

#include <cuda_runtime.h>

#include <algorithm>
#include <math.h>
#include <mutex>

#include "kernels.h"
#include "pagedkv.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int kPartitionQuantum = 32;    // partitions are whole pipeline stages
constexpr int kMaxAutoPartition = 2048;  // longest partition the library picks
constexpr int kAssumedSms = 152;         // used only when no device can be queried
constexpr int kAssumedCtasPerSm = 3;

// Sticky per-device record of problems the kernels saw (PKV_DEV_* bits).
__device__ unsigned int g_device_status;

thread_local int g_last_cuda_error = 0;

std::mutex g_mutex;
unsigned int* g_status_ptr[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};

pkv_status_t cuda_fail(cudaError_t err) {
  g_last_cuda_error = static_cast<int>(err);
  return PKV_ERR_CUDA;
}

// Device address of the status word on the current device (host code may not
// take the symbol's address directly: that is a host-side shadow).
cudaError_t status_word(unsigned int** out) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    err = cudaGetSymbolAddress(&p, g_device_status);
    if (err != cudaSuccess) return err;
    g_status_ptr[dev] = static_cast<unsigned int*>(p);
  }
  *out = g_status_ptr[dev];
  return cudaSuccess;
}

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_sm_count[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    g_sm_count[dev] = n;
  }
  return g_sm_count[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_block_size(int b) { return b == 8 || b == 16 || b == 32 || b == 64 || b == 128; }

int log2_int(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

bool decode_shape_ok(int num_seqs, int num_q_heads, int num_kv_heads, int max_context_len) {
  return num_seqs >= 0 && num_q_heads > 0 && num_kv_heads > 0 &&
         num_q_heads % num_kv_heads == 0 && max_context_len >= 0;
}

// Tokens per partition when the caller leaves the choice to the library.
//
// Every partition costs a CTA start-up (barrier set-up, table window,
// pipeline fill), a drain and a round trip of its partial result through the
// workspace, so partitions are kept long (up to 2048 tokens; measured best on
// GB300 for 1k-32k contexts).  Contexts are split into whole waves of CTAs
// where a split allows it, otherwise only as far as needed to give about four
// waves.  Batches with very few (sequence, KV head) units split finer (down to
// 256 tokens) because idle SMs cost more than partition overhead there.
//
// units: CTAs per partition index ((sequence, KV head[, head chunk]) triples);
// slots: CTAs resident on the device at once; quantum: partitions are a
// multiple of it.
int partition_for(long long units, long long slots, int max_context_len, int quantum) {
  if (max_context_len <= quantum) return quantum;
  const long long target = 4 * slots;
  const int floor_tokens = units * 4 >= slots ? 1024 : 256;
  if (units < target) {
    // Prefer a split whose CTAs fill whole waves: units * p within 5 % below
    // k waves of resident CTAs, for the fewest waves k that allows a
    // partition of [floor_tokens, kMaxAutoPartition] tokens (a multiple of
    // the quantum).  On GB300 a full single wave beat the four-wave split by
    // 11 % (8 sequences x 8k tokens) and two full waves by 6 % (16 x 8k).
    for (long long k = 1; k <= 4; ++k) {
      const long long p = k * slots / units;
      if (p < 2) continue;
      long long part = (max_context_len + p - 1) / p;
      part = ((part + quantum - 1) / quantum) * quantum;
      const long long ctas = units * ((max_context_len + part - 1) / part);
      if (part < floor_tokens || part > kMaxAutoPartition || ctas > k * slots ||
          ctas * 20 < k * slots * 19)
        continue;
      return (int)part;
    }
  }
  // Otherwise split until about four waves of CTAs: on GB300 four waves beat
  // two by up to 6 % and lost nowhere on 8-64 sequences x 1k-32k tokens, the
  // last partial wave being a smaller share of the call.
  const long long parts = units >= target ? 1 : (target + units - 1) / units;
  long long part = (max_context_len + parts - 1) / parts;
  part = ((part + 255) / 256) * 256;
  if (part < floor_tokens) part = floor_tokens;
  if (part > kMaxAutoPartition) part = kMaxAutoPartition;
  if (part >= max_context_len)
    return (int)(((long long)max_context_len + quantum - 1) / quantum * quantum);
  return (int)part;
}

int device_sms() {
  const int sms = sm_count();
  return sms > 0 ? sms : kAssumedSms;  // no device: assume a GB300
}

// Partition of the CUDA-core decode kernel.
int auto_partition(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                   int max_context_len) {
  const int group = num_q_heads / num_kv_heads;
  const int gt = pkv::decode_heads_per_cta(group);
  const long long units = (long long)num_seqs * num_kv_heads * ((group + gt - 1) / gt);
  int per_sm = sm_count() > 0 ? pkv::decode_ctas_per_sm(head_dim, gt) : 0;
  if (per_sm <= 0) per_sm = kAssumedCtasPerSm;
  return partition_for(units, (long long)device_sms() * per_sm, max_context_len,
                       kPartitionQuantum);
}

// Partition of the tensor-core decode kernel.  Its CTAs are persistent and
// take the work items (sequence, KV head, partition) in turn; the launch
// uses ceil(items / rounds) CTAs for rounds = ceil(items / SMs), so every CTA
// walks the same number of items.  The choice minimises a model of the
// call's time in units of one 128-key tile streamed at an SM's share of HBM:
//   * each round takes its items' tiles times the fraction of the SMs it
//     occupies (HBM is shared), but no less than half a tile per tile, since
//     one SM streams at most about twice its share (the bytes its copy rings
//     keep in flight);
//   * each item costs about half a tile more (its output and the switch to
//     the next item), and a split about two tiles (the partials' round trip
//     and the merge).
// On GB300 this picks the fastest of the partitions measured on 8 and 64
// sequences x 1k to 8k tokens (query-head group 4) and on 32 sequences x 4k
// tokens with groups of 4 and 32: two partitions for 8 x 8k and 8 x 32k
// (64 sequence-heads, fewer than the SMs), none from 512 sequence-heads on
// (64 x 8k: 1.04 of the copy peak unsplit against 1.00 in two), none for 4k
// tokens over 256 of them, where splitting at 2k cost 4-10 %.
int tc_partition(int num_seqs, int num_kv_heads, int max_context_len) {
  const double units = (double)num_seqs * num_kv_heads;
  const double sms = (double)device_sms();
  const long long tiles = ((long long)max_context_len + pkv::kTcPartitionQuantum - 1) /
                          pkv::kTcPartitionQuantum;
  if (tiles <= 1) return pkv::kTcPartitionQuantum;
  constexpr double kMaxRate = 2.0;    // an SM alone streams about twice its share
  constexpr double kItemCost = 0.5;   // tiles per work item
  constexpr double kSplitCost = 2.0;  // tiles for a split call
  double best_cost = 0.0;
  long long best = tiles;
  // more than about eight rounds of items never pays: the search stops there
  const double most = ceil(8.0 * sms / units);
  for (long long parts = 1; parts <= tiles && (double)parts <= most; ++parts) {
    const long long pt = (tiles + parts - 1) / parts;  // tiles per partition
    if ((tiles + pt - 1) / pt != parts) continue;      // the same partition as fewer parts
    const double items = units * (double)parts;
    const double avg = (double)tiles / (double)parts;  // tiles per item
    const double rounds = ceil(items / sms);
    const double ctas = ceil(items / rounds);          // CTAs of the launch
    const double cost = rounds * avg * fmax(ctas / sms, 1.0 / kMaxRate) + rounds * kItemCost +
                        (parts > 1 ? kSplitCost : 0.0);
    if (parts == 1 || cost < best_cost) {  // ties: fewer partitions
      best_cost = cost;
      best = pt;
    }
  }
  return (int)(best * pkv::kTcPartitionQuantum);
}

// Which decode kernel runs: 0 = chosen per call, 1 = CUDA cores, 2 = tensor
// cores (where supported).  Process-wide; see pkv_set_decode_path.
int g_decode_path = 0;

// The decode kernel and partition size of one call.  The CUDA-core kernel
// streams K/V through its FMA pipes; from a group of 8 query heads on, the
// group's 2 G flops per byte exceed what those deliver at the HBM rate.  The
// tensor-core kernel (persistent, one CTA per SM, every head of the group
// per work item) leaves the threads a few instructions per key and measured
// faster than the CUDA-core one on every grouped shape of GB300 (groups of 2
// to 32, head sizes 64 and 128, 8 to 256 sequences, 1k to 32k tokens, blocks
// of 8 to 128), so it takes every grouped call it supports.  Single-head
// groups (MHA) take the CUDA-core kernel once there are enough (sequence,
// head) pairs to fill the GPU without splitting: on the OPT-13B layer (64
// sequences of lognormal lengths, 2,560 pairs) it reaches the HBM roofline,
// 0.1172 ms, where the tensor-core kernel's static walk of unequal items
// takes 0.128-0.131.  With fewer pairs the CUDA-core kernel splits the
// contexts and pays the reduction, and the tensor-core kernel measured
// faster: 2 to 16 sequences of that layer 10-50 %, 4 and 16 sequences of 4k
// tokens over 40 heads 12 and 3 %, 8 to 64 sequences of 4k tokens over 8
// heads 4-16 % (at head size 64 as well: 8-26 %); the two
// tie at 32 sequences of the layer (1,280 pairs) and at 128 of 4k tokens over
// 8 heads (1,024).
constexpr int kMhaTcPairsPerSm = 8;  // below this many pairs per SM: tensor cores

struct DecodePlan {
  bool tc;
  int partition;
};

DecodePlan decode_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                       int max_context_len, int partition_size) {
  const int group = num_q_heads / num_kv_heads;
  const int path = __atomic_load_n(&g_decode_path, __ATOMIC_RELAXED);
  const bool few_pairs =
      (long long)num_seqs * num_kv_heads < (long long)kMhaTcPairsPerSm * device_sms();
  bool tc = path == 2 || (path == 0 && (group >= 2 || few_pairs));
  if (tc && !pkv::decode_tc_supported(head_dim, group,
                                      partition_size ? partition_size
                                                     : pkv::kTcPartitionQuantum))
    tc = false;
  if (partition_size) return {tc, partition_size};
  if (!tc)
    return {false, auto_partition(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                  max_context_len)};
  return {true, tc_partition(num_seqs, num_kv_heads, max_context_len)};
}

long long num_parts_for(int max_context_len, int partition) {
  if (max_context_len <= 0) return 1;
  return (max_context_len + (long long)partition - 1) / partition;
}

}  // namespace

extern "C" {

const char* pkv_status_string(pkv_status_t status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_ERR_INVALID_ARG: return "invalid argument";
    case PKV_ERR_UNSUPPORTED: return "unsupported configuration";
    case PKV_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case PKV_ERR_OUT_OF_BLOCKS: return "out of blocks";
    case PKV_ERR_CUDA: return "CUDA error";
    case PKV_ERR_UNKNOWN_SEQ: return "unknown sequence";
    case PKV_ERR_SEQ_EXISTS: return "sequence exists";
    case PKV_ERR_TABLE_TOO_SMALL: return "block table row too small";
  }
  return "unknown status";
}

int pkv_last_cuda_error(void) { return g_last_cuda_error; }

int pkv_version(void) { return 1; }

int pkv_decode_partition_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                              int max_context_len) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len)) return -1;
  if (head_dim != 64 && head_dim != 128) return -1;
  return decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, 0).partition;
}

size_t pkv_contiguous_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int capacity, int partition_size) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, capacity)) return (size_t)-1;
  if (head_dim != 64 && head_dim != 128) return (size_t)-1;
  if (partition_size < 0 || partition_size % kPartitionQuantum) return (size_t)-1;
  const int part = partition_size ? partition_size
                                  : auto_partition(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                   capacity);
  const long long parts = num_parts_for(capacity, part);
  if (parts <= 1) return 0;
  return (size_t)num_seqs * num_q_heads * parts * (head_dim + 2) * sizeof(float);
}

int pkv_decode_uses_tensor_cores(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int max_context_len, int partition_size) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len)) return -1;
  if (head_dim != 64 && head_dim != 128) return -1;
  if (partition_size < 0 || partition_size % kPartitionQuantum) return -1;
  return decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                     partition_size).tc ? 1 : 0;
}

pkv_status_t pkv_set_decode_path(int path) {
  if (path < 0 || path > 2) return PKV_ERR_INVALID_ARG;
  __atomic_store_n(&g_decode_path, path, __ATOMIC_RELAXED);
  return PKV_OK;
}

int pkv_get_decode_path(void) { return __atomic_load_n(&g_decode_path, __ATOMIC_RELAXED); }

size_t pkv_decode_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int max_context_len, int partition_size) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len)) return (size_t)-1;
  if (head_dim != 64 && head_dim != 128) return (size_t)-1;
  if (partition_size < 0 || partition_size % kPartitionQuantum) return (size_t)-1;
  const int part = decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                               partition_size).partition;
  const long long parts = num_parts_for(max_context_len, part);
  if (parts <= 1) return 0;
  return (size_t)num_seqs * num_q_heads * parts * (head_dim + 2) * sizeof(float);
}

namespace {

// Accumulated attention weights of an attention call.
struct WeightsArgs {
  float* weights;
  int64_t stride;
  float decay;
  int window;
  void* workspace;
  size_t workspace_bytes;
};

// Contexts the calls with 32-bit position arithmetic beyond a tile take.
constexpr int kMaxPositions = 1 << 30;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// (No position, no weight: a tensor without elements has no address.)
pkv_status_t check_weights(const WeightsArgs& w, int max_context_len) {
  if ((!w.weights && max_context_len > 0) || !aligned4(w.weights) ||
      w.stride < max_context_len || !isfinite(w.decay))
    return PKV_ERR_INVALID_ARG;
  return max_context_len > kMaxPositions ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

// CTAs for the tensor-core decode kernel's persistent walk: as many as the SMs,
// or fewer so that every CTA walks the same number of items.  512 items on 152
// SMs, say, run as 4 rounds of 128 CTAs instead of 3 rounds of 152 and a fourth
// of 56; each round still keeps HBM busy (one CTA streams about twice its
// share), and no CTA waits out a short last round.
int tc_ctas(long long items) {
  const long long sms = device_sms();
  const long long rounds = (items + sms - 1) / sms;
  return rounds > 0 ? (int)std::max(1LL, (items + rounds - 1) / rounds) : 1;
}

// Workspace of the decode call with weights, in floats.  A split call: the
// partials, every partition's maximum and sum, and the step's logits; every
// call: the CTAs' own scratch for the logits of contexts of one partition.
// Rows of logits are whole 16-byte multiples.
struct DecodeWeightsLayout {
  size_t m, x, own, floats;  // offsets of ws_m, ws_x and ws_own, and the whole
  long long x_stride, own_stride;
};

DecodeWeightsLayout decode_weights_layout(int num_seqs, int num_q_heads, int num_kv_heads,
                                          int head_dim, int max_context_len, int partition) {
  DecodeWeightsLayout l{};
  const long long parts = num_parts_for(max_context_len, partition);
  const size_t pairs = (size_t)num_seqs * num_q_heads, rows = parts > 1 ? pairs * parts : 0;
  auto whole = [](long long n) { return (n + 3) / 4 * 4; };
  l.x_stride = parts > 1 ? whole(max_context_len) : 0;
  l.own_stride = whole(std::min(max_context_len, partition));
  l.m = rows * head_dim;
  l.x = whole(l.m + 2 * rows);
  l.own = l.x + pairs * l.x_stride;
  const long long ctas = tc_ctas((long long)num_seqs * num_kv_heads * parts);
  l.floats = l.own + (size_t)ctas * 2 * (num_q_heads / num_kv_heads) * l.own_stride;
  return l;
}

// Shared body of the paged decode calls.  k_new/v_new (both or neither) are
// the step's new-token rows [num_seqs, num_kv_heads, head_dim] for the fused
// append.
pkv_status_t paged_decode_impl(void* out, const void* q, const void* k_new, const void* v_new,
                               void* k_cache, void* v_cache, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* context_lens,
                               int max_context_len, int num_seqs, int num_q_heads,
                               int num_kv_heads, int head_dim, int block_size, int num_blocks,
                               float scale, pkv_dtype_t dtype, int partition_size,
                               void* workspace, size_t workspace_bytes, pkv_stream_t stream,
                               const WeightsArgs* wa = nullptr) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len))
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (partition_size < 0 || partition_size % kPartitionQuantum) return PKV_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens)) & 3u)
    return PKV_ERR_INVALID_ARG;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size < max_context_len) return PKV_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return PKV_ERR_INVALID_ARG;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return PKV_ERR_INVALID_ARG;

  const int group = num_q_heads / num_kv_heads;
  const int gt = pkv::decode_heads_per_cta(group);
  DecodePlan plan = decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                partition_size);
  if (wa) {
    const pkv_status_t st = check_weights(*wa, max_context_len);
    if (st != PKV_OK) return st;
    plan = {true, partition_size ? partition_size
                                 : tc_partition(num_seqs, num_kv_heads, max_context_len)};
    if (!pkv::decode_tc_supported(head_dim, group, plan.partition)) return PKV_ERR_UNSUPPORTED;
    if (num_parts_for(max_context_len, plan.partition) * num_kv_heads * num_seqs > 0x7fffffffLL)
      return PKV_ERR_UNSUPPORTED;  // work items are counted in 32 bits
  }
  const int head_chunks = plan.tc ? 1 : (group + gt - 1) / gt;
  const int part = plan.partition;
  const long long parts = num_parts_for(max_context_len, part);
  if (num_seqs > 65535 || (long long)num_kv_heads * head_chunks > 65535 || parts > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;
  if ((long long)num_seqs * num_q_heads > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  if (plan.tc && (long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;

  pkv::DecodeParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_new = k_new;
  p.v_new = v_new;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.head_chunks = head_chunks;
  p.block_size = block_size;
  p.log2_block = log2_int(block_size);
  p.num_blocks = num_blocks;
  p.partition_size = part;
  p.num_parts = (int)parts;
  p.qscale = scale * 1.4426950408889634f;  // log2(e): softmax is evaluated with exp2
  if (wa) {
    const DecodeWeightsLayout l = decode_weights_layout(num_seqs, num_q_heads, num_kv_heads,
                                                        head_dim, max_context_len, part);
    if (l.floats > 0 && (!workspace || workspace_bytes < l.floats * sizeof(float)))
      return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    float* ws = static_cast<float*>(workspace);
    if (parts > 1) {
      p.ws_o = ws;
      p.ws_m = ws + l.m;
      p.ws_l = p.ws_m + (size_t)num_seqs * num_q_heads * parts;
      p.ws_x = ws + l.x;
      p.x_stride = l.x_stride;
    }
    p.ws_own = ws + l.own;
    p.own_stride = l.own_stride;
    p.weights = wa->weights;
    p.weights_stride = wa->stride;
    p.decay = wa->decay;
  } else if (parts > 1) {
    const size_t need = (size_t)num_seqs * num_q_heads * parts * (head_dim + 2) * sizeof(float);
    if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    float* ws = static_cast<float*>(workspace);
    const size_t rows = (size_t)num_seqs * num_q_heads * parts;
    p.ws_o = ws;
    p.ws_m = ws + rows * head_dim;
    p.ws_l = p.ws_m + rows;
  }
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  if (plan.tc) {
    bool unsupported = false;
    const int ctas = tc_ctas(parts * num_kv_heads * (long long)num_seqs);
    err = pkv::launch_paged_decode_tc(p, dtype, head_dim, ctas,
                                      reinterpret_cast<cudaStream_t>(stream), &unsupported);
    if (unsupported) return PKV_ERR_UNSUPPORTED;
    if (wa && err == cudaSuccess && parts > 1)
      err = pkv::launch_decode_weights(p, reinterpret_cast<cudaStream_t>(stream));
  } else {
    err = pkv::launch_paged_decode(p, dtype, head_dim, gt,
                                   reinterpret_cast<cudaStream_t>(stream));
  }
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

}  // namespace

pkv_status_t pkv_paged_attn_decode(void* out, const void* q, const void* k_cache,
                                   const void* v_cache, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* context_lens,
                                   int max_context_len, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int head_dim, int block_size,
                                   int num_blocks, float scale, pkv_dtype_t dtype,
                                   int partition_size, void* workspace, size_t workspace_bytes,
                                   pkv_stream_t stream) {
  // The caches are only read on this path.
  return paged_decode_impl(out, q, nullptr, nullptr, const_cast<void*>(k_cache),
                           const_cast<void*>(v_cache), block_tables, max_blocks_per_seq,
                           context_lens, max_context_len, num_seqs, num_q_heads, num_kv_heads,
                           head_dim, block_size, num_blocks, scale, dtype, partition_size,
                           workspace, workspace_bytes, stream);
}

pkv_status_t pkv_paged_attn_decode_append(void* out, const void* q, const void* k_new,
                                          const void* v_new, void* k_cache, void* v_cache,
                                          const int32_t* block_tables, int max_blocks_per_seq,
                                          const int32_t* context_lens, int max_context_len,
                                          int num_seqs, int num_q_heads, int num_kv_heads,
                                          int head_dim, int block_size, int num_blocks,
                                          float scale, pkv_dtype_t dtype, int partition_size,
                                          void* workspace, size_t workspace_bytes,
                                          pkv_stream_t stream) {
  if (num_seqs > 0 && (!k_new || !v_new)) return PKV_ERR_INVALID_ARG;
  return paged_decode_impl(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                           max_blocks_per_seq, context_lens, max_context_len, num_seqs,
                           num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                           dtype, partition_size, workspace, workspace_bytes, stream);
}

size_t pkv_decode_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                         int head_dim, int max_context_len, int partition_size) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len)) return (size_t)-1;
  if (partition_size < 0 || max_context_len > kMaxPositions) return (size_t)-1;
  const int part = partition_size ? partition_size
                                  : tc_partition(num_seqs, num_kv_heads, max_context_len);
  if (!pkv::decode_tc_supported(head_dim, num_q_heads / num_kv_heads, part)) return (size_t)-1;
  return decode_weights_layout(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, part)
             .floats * sizeof(float);
}

pkv_status_t pkv_paged_attn_decode_weights(
    void* out, float* weights, int64_t weights_stride, float decay, const void* q,
    const void* k_cache, const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    pkv_dtype_t dtype, int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream) {
  const WeightsArgs wa{weights, weights_stride, decay, 0, workspace, workspace_bytes};
  return paged_decode_impl(out, q, nullptr, nullptr, const_cast<void*>(k_cache),
                           const_cast<void*>(v_cache), block_tables, max_blocks_per_seq,
                           context_lens, max_context_len, num_seqs, num_q_heads, num_kv_heads,
                           head_dim, block_size, num_blocks, scale, dtype, partition_size,
                           workspace, workspace_bytes, stream, &wa);
}

pkv_status_t pkv_contiguous_attn_decode(void* out, const void* q, const void* k_cache,
                                        const void* v_cache, const int32_t* context_lens,
                                        int capacity, int num_seqs, int num_q_heads,
                                        int num_kv_heads, int head_dim, float scale,
                                        pkv_dtype_t dtype, int partition_size, void* workspace,
                                        size_t workspace_bytes, pkv_stream_t stream) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, capacity)) return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (partition_size < 0 || partition_size % kPartitionQuantum) return PKV_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !context_lens) return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(context_lens) & 3u) return PKV_ERR_INVALID_ARG;
  if (capacity <= 0) return PKV_ERR_INVALID_ARG;

  const int group = num_q_heads / num_kv_heads;
  const int gt = pkv::decode_heads_per_cta(group);
  const int head_chunks = (group + gt - 1) / gt;
  const int part = partition_size ? partition_size
                                  : auto_partition(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                   capacity);
  const long long parts = num_parts_for(capacity, part);
  if (num_seqs > 65535 || (long long)num_kv_heads * head_chunks > 65535 || parts > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;
  if ((long long)num_seqs * num_q_heads > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;

  pkv::DecodeParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = nullptr;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = 1;   // one "block" per sequence: its whole reservation
  p.max_context_len = capacity;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.head_chunks = head_chunks;
  p.block_size = capacity;
  p.log2_block = 0;
  p.num_blocks = num_seqs;
  p.partition_size = part;
  p.num_parts = (int)parts;
  p.qscale = scale * 1.4426950408889634f;
  if (parts > 1) {
    const size_t need = (size_t)num_seqs * num_q_heads * parts * (head_dim + 2) * sizeof(float);
    if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    float* ws = static_cast<float*>(workspace);
    const size_t rows = (size_t)num_seqs * num_q_heads * parts;
    p.ws_o = ws;
    p.ws_m = ws + rows * head_dim;
    p.ws_l = p.ws_m + rows;
  }
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_contiguous_decode(p, dtype, head_dim, gt,
                                      reinterpret_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

namespace {

// Shared body of the prompt-chunk calls.
pkv_status_t paged_prefill_impl(void* out, const void* q, int total_queries,
                                const int32_t* query_start, int max_query_len,
                                const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, int max_context_len, int num_seqs,
                                int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                int num_blocks, float scale, pkv_dtype_t dtype,
                                pkv_stream_t stream, const WeightsArgs* wa = nullptr) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len))
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!isfinite(scale) || max_query_len < 0 || total_queries < 0) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads / num_kv_heads > 128) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_query_len == 0 || total_queries == 0) return PKV_OK;
  if (!out || !q || !query_start || !k_cache || !v_cache || !block_tables || !context_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
       reinterpret_cast<uintptr_t>(query_start)) & 3u)
    return PKV_ERR_INVALID_ARG;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if ((long long)max_blocks_per_seq * block_size < max_context_len) return PKV_ERR_INVALID_ARG;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if ((long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;

  pkv::PrefillArgs a{};
  if (wa) {
    const pkv_status_t st = check_weights(*wa, max_context_len);
    if (st != PKV_OK) return st;
    if (wa->window < 0) return PKV_ERR_INVALID_ARG;
    if (!wa->workspace ||
        wa->workspace_bytes < pkv_prefill_weights_workspace_size(total_queries, num_q_heads))
      return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(wa->workspace)) return PKV_ERR_INVALID_ARG;
    a.lse = static_cast<float*>(wa->workspace);
    a.weights = wa->weights;
    a.weights_stride = wa->stride;
    a.window = wa->window;
    a.decay = wa->decay;
  }
  a.out = out;
  a.q = q;
  a.total_queries = total_queries;
  a.query_start = query_start;
  a.max_query_len = max_query_len;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.context_lens = context_lens;
  a.max_context_len = max_context_len;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale = scale;
  a.dtype = dtype;
  if (wa && pkv::prefill_weights_ctas(a) > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  cudaError_t err = status_word(&a.status);
  if (err != cudaSuccess) return cuda_fail(err);
  a.sm_count = sm_count() > 0 ? sm_count() : kAssumedSms;
  bool unsupported = false;
  err = pkv::launch_paged_prefill(a, reinterpret_cast<cudaStream_t>(stream), &unsupported);
  if (wa && err == cudaSuccess && !unsupported)
    err = pkv::launch_prefill_weights(a, reinterpret_cast<cudaStream_t>(stream), &unsupported);
  if (unsupported) return PKV_ERR_UNSUPPORTED;
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

}  // namespace

pkv_status_t pkv_paged_attn_prefill(void* out, const void* q, int total_queries,
                                    const int32_t* query_start, int max_query_len,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, int max_context_len,
                                    int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size, int num_blocks, float scale,
                                    pkv_dtype_t dtype, pkv_stream_t stream) {
  return paged_prefill_impl(out, q, total_queries, query_start, max_query_len, k_cache, v_cache,
                            block_tables, max_blocks_per_seq, context_lens, max_context_len,
                            num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                            scale, dtype, stream);
}

size_t pkv_prefill_weights_workspace_size(int total_queries, int num_q_heads) {
  if (total_queries < 0 || num_q_heads <= 0) return (size_t)-1;
  return (size_t)total_queries * num_q_heads * sizeof(float);
}

pkv_status_t pkv_paged_attn_prefill_weights(
    void* out, float* weights, int64_t weights_stride, float decay, int window, const void* q,
    int total_queries, const int32_t* query_start, int max_query_len, const void* k_cache,
    const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    pkv_dtype_t dtype, void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  const WeightsArgs wa{weights, weights_stride, decay, window, workspace, workspace_bytes};
  return paged_prefill_impl(out, q, total_queries, query_start, max_query_len, k_cache, v_cache,
                            block_tables, max_blocks_per_seq, context_lens, max_context_len,
                            num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                            scale, dtype, stream, &wa);
}

pkv_status_t pkv_rope_kv_append(void* q_out, int64_t q_out_stride, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int32_t* positions,
                                const double* inv_freq, int rot_dim, int interleaved,
                                float attn_factor, void* k_cache, void* v_cache,
                                const int64_t* slot_mapping, int num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                pkv_dtype_t dtype, pkv_stream_t stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!isfinite(attn_factor)) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !k || !v || !positions || !inv_freq || !k_cache || !v_cache || !slot_mapping)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(positions))
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(inv_freq) | reinterpret_cast<uintptr_t>(slot_mapping)) & 7u)
    return PKV_ERR_INVALID_ARG;
  if ((q_out_stride | q_stride | k_stride | v_stride) % 8) return PKV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (q_out_stride < q_row || q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
    return PKV_ERR_INVALID_ARG;
  if (q_out == q && q_out_stride != q_stride) return PKV_ERR_INVALID_ARG;
  pkv::RopeParams p{};
  p.q_out = q_out;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out_stride = q_out_stride;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.slot_mapping = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.num_slots = (long long)num_blocks * block_size;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0;
  p.factor = attn_factor;
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_rope_kv_append(p, num_tokens, dtype, reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

pkv_status_t pkv_kv_evict_select(int32_t* keep, int32_t* new_lens, const float* weights,
                                 int64_t weights_stride, const int32_t* context_lens,
                                 int max_context_len, int num_seqs, int num_kv_heads, int budget,
                                 int recent, int sinks, pkv_stream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || max_context_len < 0 || budget <= 0 || recent < 0 ||
      sinks < 0 || (int64_t)recent + sinks > budget || weights_stride < max_context_len)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs > 65535 || num_kv_heads > 65535 || max_context_len > kMaxPositions ||
      budget > kMaxPositions)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!keep || (!weights && max_context_len > 0) || !context_lens) return PKV_ERR_INVALID_ARG;
  if (new_lens == context_lens) return PKV_ERR_INVALID_ARG;  // other heads still read it
  if (!aligned4(keep) || !aligned4(new_lens) || !aligned4(weights) || !aligned4(context_lens))
    return PKV_ERR_INVALID_ARG;
  pkv::SelectParams p{};
  p.keep = keep;
  p.new_lens = new_lens;
  p.weights = weights;
  p.context_lens = context_lens;
  p.weights_stride = weights_stride;
  p.num_kv_heads = num_kv_heads;
  p.max_context_len = max_context_len;
  p.budget = budget;
  p.recent = recent;
  p.sinks = sinks;
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_kv_evict_select(p, num_seqs, device_sms(), reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

pkv_status_t pkv_kv_compact(void* k_cache, void* v_cache, float* weights, int64_t weights_stride,
                            const int32_t* src_tables, int max_blocks_per_seq,
                            const int32_t* dst_tables, int dst_blocks_per_seq,
                            const int32_t* keep, int budget, const int32_t* context_lens,
                            int max_context_len, int num_seqs, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, pkv_dtype_t dtype,
                            pkv_stream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || max_context_len < 0 || budget <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535 || max_context_len > kMaxPositions ||
      budget > kMaxPositions)
    return PKV_ERR_UNSUPPORTED;
  if (max_blocks_per_seq <= 0 || dst_blocks_per_seq <= 0 ||
      (long long)max_blocks_per_seq * block_size < max_context_len ||
      (long long)dst_blocks_per_seq * block_size < std::min(budget, max_context_len))
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !src_tables || !dst_tables || !keep || !context_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(src_tables) ||
      !aligned4(dst_tables) || !aligned4(keep) || !aligned4(context_lens))
    return PKV_ERR_INVALID_ARG;
  if (weights && (!aligned4(weights) || weights_stride < max_context_len))
    return PKV_ERR_INVALID_ARG;
  pkv::CompactParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.weights = weights;
  p.src_tables = src_tables;
  p.dst_tables = dst_tables;
  p.keep = keep;
  p.context_lens = context_lens;
  p.weights_stride = weights_stride;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.dst_blocks_per_seq = dst_blocks_per_seq;
  p.max_len = max_context_len;
  p.budget = budget;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.log2_block = log2_int(block_size);
  p.num_blocks = num_blocks;
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_kv_compact(p, num_seqs, device_sms(), reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

namespace {

// The caches of a call over 8-bit rows.
bool fp8_cache_ok(const void* k_cache, const void* v_cache, const void* k_scales,
                  const void* v_scales) {
  return k_cache && v_cache && k_scales && v_scales && aligned16(k_cache) && aligned16(v_cache) &&
         aligned16(k_scales) && aligned16(v_scales);
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

}  // namespace

pkv_status_t pkv_kv_append_fp8(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, pkv_dtype_t dtype,
                               pkv_stream_t stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if ((k_stride | v_stride) % 8 || k_stride < row || v_stride < row) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !aligned16(k) || !aligned16(v) || !aligned8(slot_mapping) ||
      !fp8_cache_ok(k_cache, v_cache, k_scales, v_scales))
    return PKV_ERR_INVALID_ARG;
  if (row / 16 > pkv::kMaxFp8Parts / num_tokens) return PKV_ERR_UNSUPPORTED;
  pkv::AppendFp8Params p{};
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = static_cast<uint16_t*>(k_scales);
  p.v_scales = static_cast<uint16_t*>(v_scales);
  p.slot_mapping = slot_mapping;
  p.num_slots = (long long)num_blocks * block_size;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_kv_append_fp8(p, num_tokens, head_dim, dtype,
                                  reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

pkv_status_t pkv_block_read_fp8(void* k_out, void* v_out, int num_out_blocks, const void* k_cache,
                                const void* v_cache, const void* k_scales, const void* v_scales,
                                const int64_t* src_dst_pairs, int num_pairs, int num_kv_heads,
                                int head_dim, int block_size, int num_blocks, pkv_dtype_t dtype,
                                pkv_stream_t stream) {
  if (num_pairs < 0 || num_kv_heads <= 0 || num_blocks <= 0 || num_out_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_pairs == 0) return PKV_OK;
  if (!k_out || !v_out || !src_dst_pairs || !aligned16(k_out) || !aligned16(v_out) ||
      !aligned8(src_dst_pairs) || !fp8_cache_ok(k_cache, v_cache, k_scales, v_scales))
    return PKV_ERR_INVALID_ARG;
  if ((long long)num_kv_heads * block_size * head_dim / 16 > pkv::kMaxFp8Parts / num_pairs)
    return PKV_ERR_UNSUPPORTED;
  pkv::ReadFp8Params p{};
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = static_cast<const uint16_t*>(k_scales);
  p.v_scales = static_cast<const uint16_t*>(v_scales);
  p.pairs = src_dst_pairs;
  p.num_blocks = num_blocks;
  p.num_out_blocks = num_out_blocks;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_block_read_fp8(p, num_pairs, head_dim, dtype,
                                   reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

pkv_status_t pkv_qk_norm_rope(void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                              const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* q_weight, const void* k_weight, float eps,
                              const int32_t* positions, int64_t positions_stride, int num_axes,
                              const uint8_t* pair_axes, const double* inv_freq, int rot_dim,
                              int interleaved, float attn_factor, int num_tokens, int num_q_heads,
                              int num_kv_heads, int head_dim, pkv_dtype_t dtype,
                              pkv_stream_t stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0) return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!isfinite(attn_factor) || !isfinite(eps) || eps < 0.f) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2) return PKV_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > 255 || positions_stride < num_tokens) return PKV_ERR_INVALID_ARG;
  pkv::NormRopeParams p{};
  static_assert(pkv::kMaxRopePairs == 64, "pairs of a head of 128");
  for (int i = 0; pair_axes && i < rot_dim / 2; ++i) {
    if (pair_axes[i] >= num_axes) return PKV_ERR_INVALID_ARG;
    p.pair_axes[i] = pair_axes[i];
  }
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !k_out || !q || !k || !positions || !inv_freq) return PKV_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(k_out) || !aligned16(q) || !aligned16(k) ||
      !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(positions) || !aligned8(inv_freq))
    return PKV_ERR_INVALID_ARG;
  if ((q_out_stride | k_out_stride | q_stride | k_stride) % 8) return PKV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)num_q_heads * head_dim, k_row = (int64_t)num_kv_heads * head_dim;
  if (q_out_stride < q_row || q_stride < q_row || k_out_stride < k_row || k_stride < k_row)
    return PKV_ERR_INVALID_ARG;
  if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride))
    return PKV_ERR_INVALID_ARG;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q = q;
  p.k = k;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.positions = positions;
  p.positions_stride = positions_stride;
  p.inv_freq = inv_freq;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0;
  p.eps = eps;
  p.factor = attn_factor;
  const cudaError_t err = pkv::launch_qk_norm_rope(p, num_tokens, head_dim, dtype, device_sms(),
                                                   reinterpret_cast<cudaStream_t>(stream));
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

namespace {

struct Fp8Plan {
  int chunks;     // work items of up to pkv::kFp8Rows query rows per (sequence, KV head, partition)
  int partition;
  long long parts;
};

// Tiles per partition for `units` (sequence, KV head, chunk of rows) triples of
// `rows` query rows each over contexts of `tiles` tiles: the split that a model of
// the call's time, in us, finds shortest on the CTAs that the device holds (two
// per SM up to 32 rows, else one):
//   * an item takes its tiles and two more (its start and its output), 1.5 us each,
//     in as many rounds as the items fill; a round that leaves CTAs out is shorter,
//     to 0.8 of a full one at the least (the rest have HBM and their SM to themselves);
//   * a split call takes 7 us for the launch that joins the partial outputs, their
//     bytes, written and read, and 0.2 us a partition (a warp goes through a row's
//     partitions one after another).
// The numbers are a fit to all splits of 456 calls (1-512 units of 1-64 rows, head_dim
// 64 and 128, contexts of 1,024-65,536), but for the 7: on the device 3 fit, but
// a split costs the host a launch more and, where the caller brings no workspace, that
// (four chains of drafts over up to 600 positions, split, 28 us a call for 14).
// With 3, what the model chooses takes 1.02 times the fastest on the device in the
// mean (1.15 at most), no split 1.9 times; with 7 it leaves contexts of 1,024 whole
// (1.11 there), longer ones as with 3.  Constants by classes of rows and no time per
// partition: 1.06 and 1.75.  For example (us, the
// chosen one first): 4 x 16,384 positions, 8 heads of 64 rows, 32 tiles 64, 15 tiles
// 70, unsplit 178; 1 x 65,536, one head of 4 rows, 9 tiles 25, 3 tiles 39, unsplit 364.
// Above 16 partitions the search takes steps of a sixteenth, and the numbers that fill
// one, two and three rounds (66 evaluations at most; all of them choose no better).
long long fp8_partition_tiles(long long units, long long rows, int head_dim, long long tiles) {
  constexpr double kTileUs = 1.5, kItemTiles = 2.0, kLeast = 0.8, kJoinUs = 7.0, kPartUs = 0.2;
  const long long slots = (rows > 32 ? 1 : 2) * (long long)device_sms();
  const double part_us =
      kPartUs + (double)units * (double)std::min<long long>(rows, pkv::kFp8Rows) * head_dim * 8.0 / 6.8e6;
  // more than about three rounds of items never pays: the search stops there
  const long long most = std::min(tiles, 3 * slots / units + 1);
  double best_us = 0.0;
  long long best = tiles;
  for (long long parts = 1; parts <= most;) {
    const long long pt = (tiles + parts - 1) / parts, real = (tiles + pt - 1) / pt;
    const long long items = units * real, rest = items % slots;
    const double rounds = (double)(items / slots) + (rest ? fmax((double)rest / slots, kLeast) : 0.0);
    const double us = kTileUs * ((double)pt + kItemTiles) * rounds +
                      (real > 1 ? kJoinUs + (double)real * part_us : 0.0);
    if (parts == 1 || us < best_us) {
      best_us = us;
      best = pt;
    }
    // (more parts than these with the same partition are the same split)
    long long next = std::max(parts + 1 + parts / 16, real + 1);
    for (long long k = 1; k <= 3; ++k) {
      const long long full = k * slots / units;
      if (parts < full && full < next) next = full;
    }
    parts = next;
  }
  return best;
}

// The split of a call over an 8-bit cache; false for sizes it does not take.
bool fp8_plan(int total_queries, int max_query_len, int num_seqs, int num_q_heads,
              int num_kv_heads, int head_dim, int max_context_len, int partition_size,
              Fp8Plan* plan) {
  if (head_dim != 64 && head_dim != 128) return false;
  if (max_query_len > pkv::kMaxDrafts || max_context_len > kMaxPositions) return false;
  if ((long long)total_queries * num_q_heads > 0x7fffffffLL) return false;
  const long long rows = (long long)std::max(max_query_len, 1) * (num_q_heads / num_kv_heads);
  const long long chunks = (rows + pkv::kFp8Rows - 1) / pkv::kFp8Rows;
  if (num_kv_heads > 65535 || num_seqs > 65535 || chunks > 65535) return false;
  const long long units = chunks * num_kv_heads * std::max(num_seqs, 1);
  if (units > 0x7fffffffLL) return false;
  plan->chunks = (int)chunks;
  plan->partition = partition_size;
  if (partition_size == 0) {
    constexpr int kQuantum = pkv::kTcPartitionQuantum;
    const long long tiles = std::max(1, (max_context_len + kQuantum - 1) / kQuantum);
    plan->partition =
        (int)(fp8_partition_tiles(units, rows, head_dim, tiles) * kQuantum);
  }
  plan->parts = num_parts_for(max_context_len, plan->partition);
  return plan->parts <= 0x7fffffffLL / units;
}

size_t fp8_workspace(int total_queries, int num_q_heads, int head_dim, const Fp8Plan& plan) {
  return plan.parts > 1 ? (size_t)total_queries * num_q_heads * plan.parts * (head_dim + 2) *
                              sizeof(float)
                        : 0;
}

// Shared body of the attention calls over an 8-bit cache; query_start is
// nullptr for one query per sequence.
pkv_status_t attn_fp8_impl(void* out, const void* q, int total_queries, const int32_t* query_start,
                           int max_query_len, const int64_t* tree_masks, const void* k_cache,
                           const void* v_cache, const void* k_scales, const void* v_scales,
                           const int32_t* block_tables, int max_blocks_per_seq,
                           const int32_t* context_lens, int max_context_len, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, float scale, pkv_dtype_t dtype, int partition_size,
                           void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len) ||
      total_queries < 0 || max_query_len < 0)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (partition_size < 0 || partition_size % pkv::kTcPartitionQuantum) return PKV_ERR_INVALID_ARG;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  Fp8Plan plan;
  if (!fp8_plan(total_queries, max_query_len, num_seqs, num_q_heads, num_kv_heads, head_dim,
                max_context_len, partition_size, &plan))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_queries == 0 || max_query_len == 0) return PKV_OK;
  if (!out || !q || !block_tables || !context_lens || !aligned16(out) || !aligned16(q) ||
      !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start) ||
      !aligned8(tree_masks) || !fp8_cache_ok(k_cache, v_cache, k_scales, v_scales))
    return PKV_ERR_INVALID_ARG;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0 ||
      (long long)max_blocks_per_seq * block_size < max_context_len)
    return PKV_ERR_INVALID_ARG;
  if ((long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  if (workspace_bytes < fp8_workspace(total_queries, num_q_heads, head_dim, plan) ||
      (plan.parts > 1 && !workspace))
    return PKV_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
  pkv::AttnFp8Params p{};
  p.out = out;
  p.q = q;
  p.query_start = query_start;
  p.tree_masks = tree_masks;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = static_cast<const uint16_t*>(k_scales);
  p.v_scales = static_cast<const uint16_t*>(v_scales);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.max_query_len = max_query_len;
  p.total_queries = total_queries;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.qscale = scale * 1.4426950408889634f;  // log2(e): softmax is evaluated with exp2
  p.sms = device_sms();
  p.chunks = plan.chunks;
  p.partition_size = plan.partition;
  p.num_parts = (int)plan.parts;
  if (plan.parts > 1) {
    const size_t rows = (size_t)total_queries * num_q_heads * plan.parts;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_m = p.ws_o + rows * head_dim;
    p.ws_l = p.ws_m + rows;
  }
  cudaError_t err = status_word(&p.status);
  if (err != cudaSuccess) return cuda_fail(err);
  bool unsupported = false;
  err = pkv::launch_attn_fp8(p, head_dim, dtype, reinterpret_cast<cudaStream_t>(stream),
                             &unsupported);
  if (unsupported) return PKV_ERR_UNSUPPORTED;
  return err != cudaSuccess ? cuda_fail(err) : PKV_OK;
}

}  // namespace

pkv_status_t pkv_paged_attn_decode_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache, const void* k_scales,
    const void* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    pkv_dtype_t dtype, int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream) {
  return attn_fp8_impl(out, q, num_seqs, nullptr, 1, nullptr, k_cache, v_cache, k_scales, v_scales,
                       block_tables, max_blocks_per_seq, context_lens, max_context_len, num_seqs,
                       num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, dtype,
                       partition_size, workspace, workspace_bytes, stream);
}

pkv_status_t pkv_paged_attn_tree_fp8(
    void* out, const void* q, int total_queries, const int32_t* query_start, int max_query_len,
    const int64_t* tree_masks, const void* k_cache, const void* v_cache, const void* k_scales,
    const void* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    pkv_dtype_t dtype, int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream) {
  if (num_seqs > 0 && total_queries > 0 && (!query_start || !tree_masks))
    return PKV_ERR_INVALID_ARG;
  return attn_fp8_impl(out, q, total_queries, query_start, max_query_len, tree_masks, k_cache,
                       v_cache, k_scales, v_scales, block_tables, max_blocks_per_seq, context_lens,
                       max_context_len, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, scale, dtype, partition_size, workspace, workspace_bytes,
                       stream);
}

size_t pkv_decode_fp8_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                     int max_context_len, int partition_size) {
  return pkv_tree_fp8_workspace_size(num_seqs, 1, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                     max_context_len, partition_size);
}

size_t pkv_tree_fp8_workspace_size(int total_queries, int max_query_len, int num_seqs,
                                   int num_q_heads, int num_kv_heads, int head_dim,
                                   int max_context_len, int partition_size) {
  Fp8Plan plan;
  if (!decode_shape_ok(num_seqs, num_q_heads, num_kv_heads, max_context_len) ||
      total_queries < 0 || max_query_len < 0 || partition_size < 0 ||
      partition_size % pkv::kTcPartitionQuantum ||
      !fp8_plan(total_queries, max_query_len, num_seqs, num_q_heads, num_kv_heads, head_dim,
                max_context_len, partition_size, &plan))
    return (size_t)-1;
  return fp8_workspace(total_queries, num_q_heads, head_dim, plan);
}

pkv_status_t pkv_kv_append(const void* k, const void* v, void* k_cache, void* v_cache,
                           const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, pkv_dtype_t dtype,
                           pkv_stream_t stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (!supported_block_size(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return PKV_ERR_INVALID_ARG;
  if ((long long)num_tokens * num_kv_heads * head_dim * 2 / 16 > pkv::kMaxAppendChunks)
    return PKV_ERR_UNSUPPORTED;
  unsigned int* status = nullptr;
  cudaError_t err = status_word(&status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_kv_append(k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads,
                              head_dim, block_size, num_blocks, status,
                              reinterpret_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

pkv_status_t pkv_block_copy(void* k_cache, void* v_cache, const int64_t* src_dst_pairs,
                            int num_pairs, int num_blocks, size_t block_bytes,
                            pkv_stream_t stream) {
  if (num_pairs < 0 || num_blocks <= 0 || block_bytes == 0 || block_bytes % 16)
    return PKV_ERR_INVALID_ARG;
  if (num_pairs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !src_dst_pairs) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(src_dst_pairs) & 7u) return PKV_ERR_INVALID_ARG;
  unsigned int* status = nullptr;
  cudaError_t err = status_word(&status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_block_copy(k_cache, v_cache, src_dst_pairs, num_pairs, num_blocks,
                               block_bytes, status, reinterpret_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

pkv_status_t pkv_device_status(uint32_t* flags, int clear, pkv_stream_t stream) {
  unsigned int* status = nullptr;
  cudaError_t err = status_word(&status);
  if (err != cudaSuccess) return cuda_fail(err);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  err = cudaStreamSynchronize(st);
  if (err != cudaSuccess) return cuda_fail(err);
  if (flags) {
    unsigned int host = 0;
    err = cudaMemcpyAsync(&host, status, sizeof(host), cudaMemcpyDeviceToHost, st);
    if (err == cudaSuccess) err = cudaStreamSynchronize(st);
    if (err != cudaSuccess) return cuda_fail(err);
    *flags = host;
  }
  if (clear) {
    err = cudaMemsetAsync(status, 0, sizeof(unsigned int), st);
    if (err == cudaSuccess) err = cudaStreamSynchronize(st);
    if (err != cudaSuccess) return cuda_fail(err);
  }
  return PKV_OK;
}

pkv_status_t pkv_debug_wait_timeout(pkv_stream_t stream) {
  unsigned int* status = nullptr;
  cudaError_t err = status_word(&status);
  if (err != cudaSuccess) return cuda_fail(err);
  err = pkv::launch_wait_probe(status, reinterpret_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_fail(err);
  return PKV_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free decode.
//
// Some callers cannot hand this library a workspace: serving engines that
// reserve all device memory for their own pool up front and do not let a
// library allocate while it runs, and latency-critical loops where a
// cudaMalloc (which may synchronise the device) is not allowed.  For them,
// pkv_paged_attn_decode_noalloc runs the same decode with its split-context
// partials kept in a fixed array that lives in this library's device image.
// Every GPU that loads the library holds this array until the process exits.

static __device__ __align__(256) unsigned char g_noalloc_scratch[PKV_NOALLOC_SCRATCH_BYTES];

namespace {

void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the array on the current device.  Host code only sees a
// host-side stand-in under the array's name, so the address is looked up once
// per device (with that device current) and cached.
cudaError_t noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    err = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (err != cudaSuccess) return err;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" pkv_status_t pkv_paged_attn_decode_noalloc(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype, int partition_size,
    pkv_stream_t stream) {
  const size_t need = pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                max_context_len, partition_size);
  if (need == (size_t)-1) {
    // Invalid sizes: the regular entry point reports the precise error
    // before it touches any memory.
    return pkv_paged_attn_decode(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                 context_lens, max_context_len, num_seqs, num_q_heads,
                                 num_kv_heads, head_dim, block_size, num_blocks, scale, dtype,
                                 partition_size, nullptr, 0, stream);
  }
  if (need > PKV_NOALLOC_SCRATCH_BYTES) return PKV_ERR_WORKSPACE_TOO_SMALL;
  void* scratch = nullptr;
  if (need > 0) {
    const cudaError_t err = noalloc_scratch(&scratch);
    if (err != cudaSuccess) return cuda_fail(err);
  }
  // The partials need no clearing: every partition writes its slot before
  // the reduction reads it, so what an earlier call left behind is ignored.
  return pkv_paged_attn_decode(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                               context_lens, max_context_len, num_seqs, num_q_heads, num_kv_heads,
                               head_dim, block_size, num_blocks, scale, dtype, partition_size,
                               scratch, need > 0 ? (size_t)PKV_NOALLOC_SCRATCH_BYTES : 0, stream);
}
