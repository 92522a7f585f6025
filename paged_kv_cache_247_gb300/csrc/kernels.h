// Host-side launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

// The partitions of a context, in 32 bits: any int32 partition size is taken, so
// that ctx + partition and t_begin + partition may pass 2^31 (not 2^32).
__host__ __device__ inline int context_partitions(int ctx, int partition) {
  return (int)(((unsigned)ctx + (unsigned)partition - 1u) / (unsigned)partition);
}

// End of the partition that starts at t_begin (the context's, where that is
// earlier).
__host__ __device__ inline int partition_end(int ctx, int t_begin, int partition) {
  const unsigned end = (unsigned)t_begin + (unsigned)partition;
  return (unsigned)ctx < end ? ctx : (int)end;
}

// Everything one paged decode launch needs.  Filled and checked by the API
// layer; the kernels trust it.
struct DecodeParams {
  void* out;                  // [S, Hq, D] element type
  const void* q;              // [S, Hq, D]
  const void* k_cache;        // [NB, Hkv, B, D]
  const void* v_cache;        // [NB, Hkv, B, D]
  const void* k_new;          // fused append only: [S, Hkv, D] rows of position ctx - 1
  const void* v_new;          // (nullptr: plain decode)
  const int32_t* block_tables;  // [S, max_blocks_per_seq]
  const int32_t* context_lens;  // [S]
  float* ws_o;                // split only: [S, Hq, num_parts, D]
  float* ws_m;                // split only: [S, Hq, num_parts] (log2 domain)
  float* ws_l;                // split only: [S, Hq, num_parts]
  unsigned int* status;       // device status word
  int max_blocks_per_seq;
  int max_context_len;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int group;        // Hq / Hkv
  int head_chunks;  // CTAs per KV head (ceil(group / heads per CTA))
  int block_size;
  int log2_block;
  int num_blocks;
  int partition_size;  // tokens per CTA (multiple of 32)
  int num_parts;       // ceil(max_context_len / partition_size), >= 1
  float qscale;        // scale * log2(e): logits are kept in base-2 units
  // Accumulated attention weights (weights == nullptr: none; tensor-core kernel
  // only).
  float* ws_x;             // split contexts: base-2 logits [S, Hq, x_stride]
  long long x_stride;
  float* ws_own;           // unsplit ones: [CTAs, 2, group, own_stride], used in turn
  long long own_stride;
  float* weights;          // [S, Hkv, weights_stride]
  long long weights_stride;
  float decay;
};

// Query heads one CTA processes for a group size (1, 2 or 4).
int decode_heads_per_cta(int group);

// Decode CTAs resident per SM on the current device (0 if unknown).
int decode_ctas_per_sm(int head_dim, int heads_per_cta);

// Shared memory one decode CTA uses.
size_t decode_smem_bytes(int head_dim, int heads_per_cta);

// Launch the decode kernel and, when num_parts > 1, the reduction kernel.
cudaError_t launch_paged_decode(const DecodeParams& p, int dtype, int head_dim,
                                int heads_per_cta, cudaStream_t stream);

// Only the split reduction (merging num_parts partials per (sequence, query
// head)); used after the tensor-core decode kernel.
cudaError_t launch_decode_reduce(const DecodeParams& p, int dtype, int head_dim,
                                 cudaStream_t stream);

// Decode on the tensor cores: head size 64 or 128, groups of
// kMinTcGroup..kMaxTcGroup query heads (grouped heads by default, single
// heads when forced), partitions of whole 128-key tiles.
constexpr int kMinTcGroup = 1;
constexpr int kMaxTcGroup = 32;
constexpr int kTcPartitionQuantum = 128;
bool decode_tc_supported(int head_dim, int group, int partition_size);

// Persistent: min(work items, sms) CTAs, one per SM.  unsupported is set when
// the tensor maps of the caches or of q cannot be encoded.
cudaError_t launch_paged_decode_tc(const DecodeParams& p, int dtype, int head_dim, int sms,
                                   cudaStream_t stream, bool* unsupported);

// Same kernels over a contiguous cache [S, Hkv, capacity, D]: block_size is
// the capacity, block_tables is unused and sequence s reads rows of s.
cudaError_t launch_contiguous_decode(const DecodeParams& p, int dtype, int head_dim,
                                     int heads_per_cta, cudaStream_t stream);

// Multi-query (chunked prompt) attention over the paged cache.
struct PrefillArgs {
  void* out;
  const void* q;
  int total_queries;  // rows of q and out
  const int32_t* query_start;
  int max_query_len;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* context_lens;
  int max_context_len;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  int block_size;
  int num_blocks;
  float scale;
  int dtype;
  unsigned int* status;
  int sm_count;  // SMs of the device (sizes the launch order's groups)
  float* lse;    // base-2 log-sum of each row [total_queries, Hq] (nullptr: not wanted)
  float* weights;  // accumulated attention weights [S, Hkv, weights_stride]
  long long weights_stride;
  int window;      // last queries of a chunk that count (0: all)
  float decay;
};

// unsupported is set when the tensor maps of q or of the caches cannot be
// encoded, or the work needs more CTAs than a 1-D grid holds.
cudaError_t launch_paged_prefill(const PrefillArgs& a, cudaStream_t stream, bool* unsupported);

// Accumulated attention weights of a decode step from ws_x, ws_m and ws_l.
cudaError_t launch_decode_weights(const DecodeParams& p, cudaStream_t stream);

struct PrefillWeightsParams {
  const float* lse;
  float* weights;
  long long weights_stride;
  float decay;
  int window;
  const int32_t* query_start;
  const int32_t* context_lens;
  const int32_t* block_tables;
  unsigned int* status;
  int max_blocks_per_seq;
  int max_context_len;
  int num_q_heads;
  int num_kv_heads;
  int group;
  int group_pow2;
  int block_size;
  int num_blocks;
  int total_queries;
  float qscale;
  int key_tiles;
};

// CTAs of launch_prefill_weights: a call of more than 2^31 - 1 has to be refused
// before its attention is launched.
long long prefill_weights_ctas(const PrefillArgs& a);

// Accumulated attention weights of a prompt chunk, after launch_paged_prefill
// with a.lse set.
cudaError_t launch_prefill_weights(const PrefillArgs& a, cudaStream_t stream, bool* unsupported);

// Rotary positions with append.  Strides are in elements, between tokens.
struct RopeParams {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  long long q_out_stride, q_stride, k_stride, v_stride;
  const int32_t* positions;
  const double* inv_freq;  // [rot_dim / 2]
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  unsigned int* status;
  long long num_slots;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  int block_size;
  int rot_dim;
  int interleaved;
  float factor;
};

cudaError_t launch_rope_kv_append(const RopeParams& p, int num_tokens, int dtype,
                                  cudaStream_t stream);

struct SelectParams {
  int32_t* keep;           // [S, Hkv, budget]
  int32_t* new_lens;       // [S] or nullptr
  const float* weights;    // [S, Hkv, weights_stride]
  const int32_t* context_lens;
  unsigned int* status;
  long long weights_stride;
  int num_kv_heads;
  int max_context_len;
  int budget;
  int recent;
  int sinks;
  int cluster;             // CTAs per row (set by the launch)
};

cudaError_t launch_kv_evict_select(SelectParams p, int num_seqs, int sm_count,
                                   cudaStream_t stream);

struct CompactParams {
  void* k_cache;
  void* v_cache;
  float* weights;          // [S, Hkv, weights_stride] or nullptr
  const int32_t* src_tables;
  const int32_t* dst_tables;
  const int32_t* keep;     // [S, Hkv, budget]
  const int32_t* context_lens;
  unsigned int* status;
  long long weights_stride;
  int max_blocks_per_seq;  // row strides of the two tables
  int dst_blocks_per_seq;
  int max_len;             // positions the source table and the weights rows hold
  int budget;
  int num_kv_heads;
  int head_dim;
  int block_size;
  int log2_block;
  int num_blocks;
};

cudaError_t launch_kv_compact(const CompactParams& p, int num_seqs, int sm_count,
                              cudaStream_t stream);

// kv_append indexes (token, 16-byte chunk) pairs with 32 bits: a call may move
// at most this many chunks of K (and as many of V), 32 GiB each.
constexpr long long kMaxAppendChunks = 1LL << 31;

cudaError_t launch_kv_append(const void* k, const void* v, void* k_cache, void* v_cache,
                             const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks,
                             unsigned int* status, cudaStream_t stream);

cudaError_t launch_block_copy(void* k_cache, void* v_cache, const int64_t* pairs,
                              int num_pairs, int num_blocks, size_t block_bytes,
                              unsigned int* status, cudaStream_t stream);

// Diagnostic: one bounded wait on an mbarrier that nothing completes; it
// gives up after the wait limit and raises PKV_DEV_WAIT_TIMEOUT.
cudaError_t launch_wait_probe(unsigned int* status, cudaStream_t stream);

}  // namespace pkv
