/*
 * pagedkv.h — C ABI of the paged KV-cache decode library (libpagedkv.so).
 *
 * The library implements the hot path of PagedAttention-style serving on one
 * GPU: single-query decode attention that walks a per-sequence block table
 * (pkv_paged_attn_decode), the scatter of each step's new K/V into its slot
 * (pkv_kv_append), block-granular copy-on-write (pkv_block_copy), and a
 * host-side refcounted block allocator that decides slots and copies
 * (pkv_alloc_*).
 *
 * Sources, cited by page title and section:
 *   [P1] "800 kilobytes per token" (shashforge.dev)
 *   [P2] "Only 20.4% of your KV cache held actual tokens: how PagedAttention
 *        put a page table inside the attention kernel" (blog.teqners.com)
 *   [P3] "The KV cache is a systems problem" (rsw.lol)
 *
 * Conventions shared by every call
 *   - Pointers named *_cache, q, out, k, v, block_tables, context_lens,
 *     slot_mapping, src_dst_pairs and workspace are DEVICE pointers owned by
 *     the caller; the library never allocates, frees or retains them.
 *     Tensors are dense row-major with the shapes given per call; q, out, k,
 *     v and both caches must be 16-byte aligned.
 *   - The KV cache is two arrays (K and V) of shape
 *     [num_blocks, num_kv_heads, block_size, head_dim]: token position t of a
 *     sequence lives in logical block t / block_size at offset
 *     t % block_size, and logical block i lives in physical block
 *     block_tables[s][i].  ([P2] "The page table, relocated into attention".)
 *   - Every device call enqueues its kernels on `stream` (a cudaStream_t;
 *     NULL is the legacy default stream) and returns without synchronising.
 *     Argument checks happen on the host before anything is enqueued; a call
 *     that returns an error has enqueued nothing.
 *   - Stream order is kept as for any kernel.  The decode, append and copy
 *     kernels, and those of the calls for a cache smaller than the history
 *     (pkv_paged_attn_prefill_weights' attention excepted), are launched with programmatic stream serialization: their
 *     blocks may be placed on the GPU while the previous kernel on the stream
 *     is still running, but each waits for that kernel to finish (and for its
 *     writes to be visible) before it reads or writes memory.  A kernel the
 *     caller launches after them without that attribute starts after they
 *     finish, as usual.
 *   - Problems only visible on the device (a block id outside the pool, a
 *     context length beyond the table, a slot beyond the pool) never fault:
 *     the offending access is skipped or redirected to block 0, the result is
 *     undefined, and a PKV_DEV_* flag is raised in a per-device status word
 *     read by pkv_device_status().
 *   - Strides given as int64_t count elements.  Accumulated attention weights
 *     are fp32 [num_seqs, num_kv_heads, >= the contexts] with weights_stride
 *     elements between rows: weights[s][h][t] belongs to position t of batch
 *     row s, whatever blocks the position lives in.  (They may be NULL where
 *     max_context_len is 0.)
 *   - The kernels never spin on another block or another launch.  Apart from
 *     the wait for the previous kernel on the stream described above, the
 *     only waits are on their own copies into shared memory, each bounded in
 *     time (PKV_DEV_WAIT_TIMEOUT).  (The blocks of a thread-block cluster,
 *     which the hardware places together, meet at cluster barriers:
 *     pkv_kv_evict_select.)
 */
#ifndef PAGEDKV_H_
#define PAGEDKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* pkv_stream_t;

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,          /* null pointer, bad size, misaligned pointer, ... */
  PKV_ERR_UNSUPPORTED = 2,          /* valid but not built: head_dim, block_size, grid limits */
  PKV_ERR_WORKSPACE_TOO_SMALL = 3,  /* split decode needs more workspace than given */
  PKV_ERR_OUT_OF_BLOCKS = 4,        /* allocator: pool exhausted, state unchanged */
  PKV_ERR_CUDA = 5,                 /* a CUDA runtime call failed, see pkv_last_cuda_error() */
  PKV_ERR_UNKNOWN_SEQ = 6,          /* allocator: sequence id not live */
  PKV_ERR_SEQ_EXISTS = 7,           /* allocator: sequence id already live */
  PKV_ERR_TABLE_TOO_SMALL = 8       /* allocator: caller's table row shorter than the sequence */
} pkv_status_t;

typedef enum { PKV_F16 = 0, PKV_BF16 = 1 } pkv_dtype_t;

/* Flags of the per-device status word (bitwise OR of everything seen since
 * the last clear). */
#define PKV_DEV_BAD_BLOCK_ID 1u     /* a table entry or copy pair outside [0, num_blocks) */
#define PKV_DEV_BAD_CONTEXT_LEN 2u  /* context_lens[s] < 0 or > max_context_len or > table row */
#define PKV_DEV_BAD_SLOT 4u         /* slot_mapping[t] >= num_blocks * block_size */
#define PKV_DEV_WAIT_TIMEOUT 8u     /* a bounded wait inside a kernel gave up (never expected) */
#define PKV_DEV_BAD_KEEP 16u        /* keep[i] < i or not a position of the sequence */

/* Human-readable name of a status code (static string). */
const char* pkv_status_string(pkv_status_t status);

/* cudaError_t of the last PKV_ERR_CUDA returned on this host thread. */
int pkv_last_cuda_error(void);

/* ABI version, bumped on any incompatible change. */
int pkv_version(void);

/* ------------------------------------------------------------------------
 * Paged single-query decode attention.
 *
 * [P2] "The page table, relocated into attention": the kernel follows each
 * sequence's block table and gathers K and V from non-contiguous physical
 * blocks; [P2] "Why the KV cache is the thing that limits your batch": each
 * decode step is a memory-bound matrix-vector product per request.
 *
 * For every sequence s < num_seqs and query head h < num_q_heads:
 *   out[s][h][:] = softmax_t( scale * q[s][h] . K_s[t][h / G] ) @ V_s[t][h / G]
 * over t < context_lens[s], where G = num_q_heads / num_kv_heads (query head
 * h reads KV head h / G) and K_s[t] = k_cache[block_tables[s][t / B]][.][t % B].
 * Logits, softmax and the weighted sum are fp32; out is rounded to dtype
 * (round to nearest even).  On the tensor-core path (groups G of 2 to 32
 * query heads by default, see pkv_set_decode_path) the softmax
 * weights are rounded to dtype before the weighted sum, which the tensor
 * core accumulates in fp32 ([P3] "Calculate bytes per token before choosing
 * a batch": groups of query heads share one KV head, and a group of G heads
 * does 2 G flops per cache byte).  A sequence with context_lens[s] == 0 gets
 * zeros.
 * Positions at or beyond context_lens[s] are never read, and neither are
 * table entries past ceil(context_lens[s] / B).
 *
 *   out           [num_seqs, num_q_heads, head_dim]            dtype, written
 *   q             [num_seqs, num_q_heads, head_dim]            dtype
 *   k_cache/v_cache [num_blocks, num_kv_heads, block_size, head_dim] dtype
 *   block_tables  int32 [num_seqs, max_blocks_per_seq] (row stride
 *                 max_blocks_per_seq); entries must lie in [0, num_blocks)
 *   context_lens  int32 [num_seqs], each in [0, max_context_len] and
 *                 <= max_blocks_per_seq * block_size
 *   max_context_len  host-side upper bound on context_lens (sizes the grid)
 *   head_dim      64 or 128;  block_size 8, 16, 32, 64 or 128
 *   scale         finite, of either sign or zero
 *   partition_size   tokens per split-context partition: 0 lets the library
 *                 choose (pkv_decode_partition_size); otherwise a positive
 *                 multiple of 32.  When ceil(max_context_len / partition_size)
 *                 > 1 the call writes per-partition partial results into
 *                 `workspace` and launches a second, reduction kernel.
 *   workspace     device scratch of at least pkv_decode_workspace_size(...)
 *                 bytes (may be NULL when that size is 0); its contents on
 *                 entry do not matter and it is not read after the call.
 *
 * Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED,
 * PKV_ERR_WORKSPACE_TOO_SMALL, PKV_ERR_CUDA (launch failure).
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_paged_attn_decode(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Fused decode step: append the step's new token, then attend.
 *
 * One decode step appends one token per sequence and attends over the whole
 * context including it ([P2] "Why the KV cache is the thing that limits your
 * batch": the cache grows token by token; [P2] "The page table, relocated
 * into attention").  This call does both in one launch: for every sequence
 * with context_lens[s] > 0 the new token is position ctx - 1 =
 * context_lens[s] - 1, its slot is
 *   block_tables[s][(ctx - 1) / B] * B + (ctx - 1) % B,
 * and the call writes k_new[s][h][:] / v_new[s][h][:] there (bit-exact, as
 * pkv_kv_append would) while the attention uses those rows directly.  The
 * result equals pkv_kv_append followed by pkv_paged_attn_decode.
 *
 *   k_new, v_new  [num_seqs, num_kv_heads, head_dim] dtype, 16-byte aligned
 *   k_cache/v_cache are written (one row per sequence and KV head)
 * The slot's block must not be shared with another sequence (do the
 * copy-on-write pkv_block_copy first, on the same stream).  Sequences with
 * context_lens[s] == 0 append nothing.  Other arguments, results, workspace
 * and errors as pkv_paged_attn_decode.
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_paged_attn_decode_append(
    void* out, const void* q, const void* k_new, const void* v_new,
    void* k_cache, void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Allocation-free decode.  (The source pages have no counterpart: this is an
 * interface for callers, not part of the method.)
 *
 * For callers that cannot provide a workspace: engines that reserve all
 * device memory for their own pool and forbid allocation while serving, and
 * latency-critical loops where cudaMalloc, which may synchronise the device,
 * is not allowed.  Same arguments and result as pkv_paged_attn_decode minus
 * the workspace: the split-context partials go to a fixed array of
 * PKV_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads
 * the library holds until the process exits.
 *
 *   - Allocates nothing (no cudaMalloc/cudaFree, no allocating library call).
 *   - Sizes whose pkv_decode_workspace_size(...) exceeds
 *     PKV_NOALLOC_SCRATCH_BYTES are rejected with PKV_ERR_WORKSPACE_TOO_SMALL
 *     before anything is enqueued; use a larger partition_size or the
 *     workspace entry point for them.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it; make
 *     that first call before any stream capture.
 *   - All calls on a device share the one array, which keeps whatever the
 *     last call left in it.  Nothing in it needs to start at zero (each
 *     partial is written before it is read), but calls that overlap on the
 *     GPU (different streams without ordering between them) race on it:
 *     order them on one stream or with events.
 * ---------------------------------------------------------------------- */
#define PKV_NOALLOC_SCRATCH_BYTES (16u << 20) /* 16 MiB */

pkv_status_t pkv_paged_attn_decode_noalloc(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, pkv_stream_t stream);

/* Partition size the library picks for partition_size == 0 on the current
 * device (depends on its SM count and on the decode kernel the call will
 * use).  Returns a positive multiple of 32, or -1 for invalid arguments. */
int pkv_decode_partition_size(int num_seqs, int num_q_heads, int num_kv_heads,
                              int head_dim, int max_context_len);

/* Which decode kernel the decode calls use, process-wide (a tuning and test
 * control; the default suits every shape measured):
 *   0  chosen per call (default): the tensor-core kernel for grouped heads
 *      (groups of 2 to 32 query heads, head_dim 64 or 128, partition_size 0
 *      or a multiple of 128) and for single-head groups (MHA) with fewer
 *      than 8 (sequence, KV head) pairs per SM; the CUDA-core kernel
 *      otherwise (MHA with more pairs, or a partition the tensor-core
 *      kernel cannot take);
 *   1  always the CUDA-core kernel;
 *   2  the tensor-core kernel wherever it can run (groups of 1 to 32, head_dim
 *      64 or 128, partition_size 0 or a multiple of 128), else the CUDA-core
 *      one.
 * Both compute the same attention within the stated tolerance.  It changes
 * the partition pkv_decode_partition_size and pkv_decode_workspace_size
 * report, so set it before sizing a workspace, and not while another host
 * thread issues decode calls.  Returns PKV_ERR_INVALID_ARG for other
 * values. */
pkv_status_t pkv_set_decode_path(int path);
int pkv_get_decode_path(void);

/* 1 if a decode call with these sizes (partition_size as in
 * pkv_paged_attn_decode) runs the tensor-core kernel under the current
 * setting, 0 if the CUDA-core kernel, -1 for invalid arguments. */
int pkv_decode_uses_tensor_cores(int num_seqs, int num_q_heads, int num_kv_heads,
                                 int head_dim, int max_context_len, int partition_size);

/* Workspace bytes pkv_paged_attn_decode needs for these sizes (0 when the
 * call will not split).  partition_size as in pkv_paged_attn_decode.
 * Layout: fp32 partial outputs [num_seqs, num_q_heads, parts, head_dim],
 * then fp32 running maxima and fp32 denominators [num_seqs, num_q_heads,
 * parts] each, parts = ceil(max_context_len / partition).  Returns
 * (size_t)-1 for invalid arguments. */
size_t pkv_decode_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                 int head_dim, int max_context_len, int partition_size);

/* ------------------------------------------------------------------------
 * Contiguous-cache decode: the baseline without a block table.
 *
 * [P3] "When the extra machinery is not worth it": keep a simple contiguous
 * cache as a baseline and compare both under identical token distributions;
 * [P2] "What the indirection costs": the paged kernel's price is the table
 * reads, extra branches and variable lengths.  This call runs the same
 * kernels over the pre-paging layout ([P2] opening section: one contiguous
 * tensor per request, reserved at its maximum length), so the difference to
 * pkv_paged_attn_decode on the same tokens is the cost of the indirection.
 *
 *   k_cache/v_cache [num_seqs, num_kv_heads, capacity, head_dim] dtype:
 *                 sequence s holds its positions t < context_lens[s] at
 *                 [s][h][t][:]; capacity is the reservation per sequence
 *   context_lens  int32 [num_seqs], each in [0, capacity]
 * It runs the CUDA-core decode kernel (and its partition choice) whatever
 * pkv_set_decode_path says, so it is the contiguous twin of
 * pkv_paged_attn_decode under setting 1; the workspace it needs is
 * pkv_contiguous_workspace_size.  Other arguments, results and errors as
 * pkv_paged_attn_decode (with max_context_len = capacity).
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_contiguous_attn_decode(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* context_lens, int capacity,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    float scale, pkv_dtype_t dtype, int partition_size,
    void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* Workspace bytes pkv_contiguous_attn_decode needs (0 when it will not
 * split); (size_t)-1 for invalid arguments. */
size_t pkv_contiguous_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int capacity, int partition_size);

/* ------------------------------------------------------------------------
 * Multi-query (chunked prompt) attention over the paged cache.
 *
 * Prompts are processed in chunks that share the step budget with decoding
 * ([P3] "Memory savings change the scheduling question"); each chunk attends
 * causally to the sequence's cached prefix and to itself, through the block
 * table ([P2] "The page table, relocated into attention").
 *
 * Sequence s brings L_s = query_start[s+1] - query_start[s] query rows
 * q[query_start[s] .. query_start[s+1]), the last L_s positions of its
 * context: query j is position p = context_lens[s] - L_s + j, and its K/V
 * (like every position < context_lens[s]) must already be in the cache
 * (pkv_kv_append).  For every query head h:
 *   out[query_start[s] + j][h] = softmax_{t <= p}(scale * q . K_s[t][h/G]) @ V_s[t][h/G]
 * Q.K and P.V run on the tensor cores (fp32 accumulation); the softmax
 * weights P are rounded to dtype before P.V, as the operand type requires.
 *
 *   q, out        [total_queries, num_q_heads, head_dim] dtype, with
 *                 total_queries >= query_start[num_seqs] (rows of either past
 *                 total_queries are neither read nor written)
 *   query_start   int32 [num_seqs + 1], non-decreasing, starting at 0
 *   max_query_len host-side bound on L_s (sizes the grid)
 *   context_lens  int32 [num_seqs] with L_s <= context_lens[s] <= max_context_len
 *   num_q_heads / num_kv_heads <= 128
 * Other arguments as pkv_paged_attn_decode.  Errors: PKV_ERR_INVALID_ARG,
 * PKV_ERR_UNSUPPORTED (also when the caches cannot be described to the
 * tensor-memory-access unit, or when num_seqs * num_kv_heads * query tiles
 * exceeds 2^31 - 1), PKV_ERR_CUDA.
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_paged_attn_prefill(
    void* out, const void* q, int total_queries, const int32_t* query_start, int max_query_len,
    const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Append new tokens' K and V into their cache slots.
 *
 * The cache grows token by token ([P2] "Why the KV cache is the thing that
 * limits your batch"); logical blocks fill left to right ([P2] "The page
 * table, relocated into attention").
 *
 * For each token t < num_tokens with slot = slot_mapping[t] >= 0 and every
 * KV head h:  k_cache[slot / B][h][slot % B][:] = k[t][h][:]  (same for V).
 * Tokens with a negative slot are skipped (padding).  A byte copy: bit-exact.
 *
 *   k, v          [num_tokens, num_kv_heads, head_dim] dtype
 *   k_cache/v_cache [num_blocks, num_kv_heads, block_size, head_dim] dtype
 *   slot_mapping  int64 [num_tokens]; flat slot = physical_block * B + offset
 * Slots must be distinct (two tokens writing one slot race).  A slot at or
 * beyond num_blocks * block_size is skipped and flags PKV_DEV_BAD_SLOT.
 * Errors: PKV_ERR_INVALID_ARG (null or misaligned pointer, negative sizes,
 * bad dtype), PKV_ERR_UNSUPPORTED (head_dim or block_size not built, or more
 * than 2^31 16-byte chunks of K in one call: 32 GiB), PKV_ERR_CUDA.
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_kv_append(
    const void* k, const void* v, void* k_cache, void* v_cache,
    const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, pkv_dtype_t dtype, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Block-granular copy-on-write.
 *
 * [P2] "The part everyone forgets: pages enable sharing, not just packing":
 * when a sample writes into a shared, partially filled block, a fresh block
 * is allocated and one block's worth of data is copied ([P1] "The old
 * answer, imported honestly": copy on write when a shared block diverges).
 *
 * For each pair i < num_pairs: copies block_bytes bytes of physical block
 * src = src_dst_pairs[2i] onto block dst = src_dst_pairs[2i+1], in k_cache
 * and in v_cache (block_bytes = num_kv_heads * block_size * head_dim *
 * element size, a multiple of 16).  Destinations must be distinct and no
 * destination may also be a source in the same call (pairs run in parallel).
 * Ids outside [0, num_blocks) skip the pair and flag PKV_DEV_BAD_BLOCK_ID.
 *
 *   src_dst_pairs int64 [num_pairs, 2], device memory
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_block_copy(
    void* k_cache, void* v_cache, const int64_t* src_dst_pairs, int num_pairs,
    int num_blocks, size_t block_bytes, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * A cache smaller than the history.
 *
 * [P3] "Eviction and reuse can move costs elsewhere": a sequence that outgrows
 * its share of the pool drops cached positions.  The calls below keep it
 * going: rotary positions applied as new rows are appended (a token's position
 * then no longer has to be its index in the cache), attention that also
 * accumulates how much weight each cached position received, the choice of
 * the positions to keep, and the move of their rows to the front, after which
 * pkv_alloc_shrink_seqs returns the blocks behind them to the pool.
 * ---------------------------------------------------------------------- */

/* Rotary positions with append, in one launch.
 *
 * For each token t with pos = positions[t] >= 0, each pair i < rot_dim / 2 of
 * every head row of q and k is turned by the angle a = pos * inv_freq[i]:
 *   first'  = attn_factor * (first cos a - second sin a)
 *   second' = attn_factor * (first sin a + second cos a)
 * with (first, second) the elements (2i, 2i + 1) if interleaved, else
 * (i, i + rot_dim / 2); elements from rot_dim on are copied.  The angle is
 * formed in 64 bits, the products in fp32, and each result is rounded once to
 * dtype.  q goes to q_out; k and v (v unturned) go to slot slot_mapping[t], as
 * pkv_kv_append.  A token with a negative position is padding: nothing is
 * written for it.  A negative slot skips k and v only.  A slot at or beyond
 * num_blocks * block_size does so too and flags PKV_DEV_BAD_SLOT.
 *
 *   q_out, q      [num_tokens, num_q_heads, head_dim] dtype, tokens *_stride
 *                 elements apart (a multiple of 8, at least a token's row, so
 *                 that slices of a joint projection need no copy); q_out may
 *                 be q with the same stride, and must not overlap it otherwise
 *   k, v          [num_tokens, num_kv_heads, head_dim] likewise
 *   positions     int32 [num_tokens]
 *   inv_freq      double [rot_dim / 2], radians per position, scaled for long
 *                 contexts as the model wants
 *   rot_dim       even, 2 .. head_dim
 *   slot_mapping  int64 [num_tokens], distinct where not negative
 * Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED (head_dim or block_size not
 * built, 65,536 heads or more), PKV_ERR_CUDA. */
pkv_status_t pkv_rope_kv_append(
    void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
    const void* k, int64_t k_stride, const void* v, int64_t v_stride,
    const int32_t* positions, const double* inv_freq, int rot_dim, int interleaved,
    float attn_factor, void* k_cache, void* v_cache, const int64_t* slot_mapping,
    int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, pkv_dtype_t dtype, pkv_stream_t stream);

/* Decode attention that accumulates attention weights: pkv_paged_attn_decode,
 * and for every KV head h and position t < context_lens[s]
 *   weights[s][h][t] = decay * weights[s][h][t] + sum_g p_g(t)
 * over the softmax weights p_g of the query heads g that read h (fp32; decay 0
 * overwrites without reading).  Positions at or beyond context_lens[s] keep
 * their values.  Runs the tensor-core kernel: groups of at most 32 query
 * heads, partition_size 0 or a multiple of 128 (PKV_ERR_UNSUPPORTED
 * otherwise; pkv_paged_attn_prefill_weights takes larger groups, one query per
 * sequence, with its tiles mostly empty: 120 us for 16 sequences of 4,096 over
 * 4 KV heads of 128 with groups of 33, whose bytes take 20), whatever
 * pkv_set_decode_path says.
 *   weights_stride  >= max_context_len
 *   workspace       pkv_decode_weights_workspace_size(...) bytes, split
 *                   context or not: the step's logits are kept there.  It grows
 *                   with max_context_len, not with the contexts: unsplit, two
 *                   rows of logits per query head of a group and CTA, 4 *
 *                   2 * CTAs * G * max_context_len bytes (at most one CTA per
 *                   SM; 67 MB for 64 sequences over 8 KV heads with groups of 8
 *                   and a bound of 8,192, 1.07 GB at 131,072); split, every
 *                   logit of the call besides.  So pass a bound near the longest
 *                   context, and keep the workspace between steps.
 * Everything else as pkv_paged_attn_decode. */
pkv_status_t pkv_paged_attn_decode_weights(
    void* out, float* weights, int64_t weights_stride, float decay,
    const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream);

/* Depends on the SM count of the current device.  (size_t)-1 for invalid
 * arguments or sizes the call does not support. */
size_t pkv_decode_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                         int head_dim, int max_context_len, int partition_size);

/* Chunked-prompt attention that accumulates attention weights:
 * pkv_paged_attn_prefill, and for every sequence with L_s > 0 queries, every
 * KV head h and position t < context_lens[s]
 *   weights[s][h][t] = decay * weights[s][h][t] + sum_j sum_g p_{j,g}(t)
 * over the last min(window, L_s) queries j (window 0: all of them) and the
 * query heads g that read h.  The sums run in a fixed order (the same bits on
 * every call).  A sequence without queries keeps its weights.
 *   weights_stride  >= max_context_len
 *   workspace       pkv_prefill_weights_workspace_size(...) bytes
 * Everything else as pkv_paged_attn_prefill. */
pkv_status_t pkv_paged_attn_prefill_weights(
    void* out, float* weights, int64_t weights_stride, float decay, int window,
    const void* q, int total_queries, const int32_t* query_start, int max_query_len,
    const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* (size_t)-1 for invalid arguments. */
size_t pkv_prefill_weights_workspace_size(int total_queries, int num_q_heads);

/* The positions to keep, per sequence and KV head.
 *
 * With n = context_lens[s]: if n <= budget, keep[s][h] = 0 .. n - 1.  Otherwise
 * the first `sinks` positions, the last `recent` ones, and of the others the
 * budget - sinks - recent with the largest weights (of equal weights the
 * lowest positions; NaN ranks below everything), in ascending order.  Entries
 * past min(n, budget) are -1.  new_lens[s] = min(n, budget) if new_lens is not
 * NULL (another array than context_lens).
 *
 *   keep          int32 [num_seqs, num_kv_heads, budget]
 *   weights       fp32, weights_stride >= max_context_len
 *   sinks, recent >= 0 with sinks + recent <= budget */
pkv_status_t pkv_kv_evict_select(
    int32_t* keep, int32_t* new_lens, const float* weights, int64_t weights_stride,
    const int32_t* context_lens, int max_context_len, int num_seqs, int num_kv_heads,
    int budget, int recent, int sinks, pkv_stream_t stream);

/* Move the kept rows of every sequence and KV head to its front.
 *
 * For i < min(context_lens[s], budget): position i of (s, h) receives the K
 * and V rows of position keep[s][h][i], read through src_tables and written
 * through dst_tables (a byte copy: bit-exact), and weights[s][h][i] receives
 * weights[s][h][keep[s][h][i]]; the weights of the positions from there to
 * context_lens[s] become 0.  keep has to ascend strictly.  An entry below its
 * index or outside the sequence is skipped and flags PKV_DEV_BAD_KEEP.
 *
 * dst_tables may be src_tables (rows move in place), or name another block
 * where a source block is shared ([P3] "Shared prefixes need ownership
 * rules"): pkv_alloc_shrink_seqs gives every shared block of the kept part a
 * fresh one.  A destination block must belong to one sequence, and must not be
 * a source block of another sequence or of another place of the same one.
 *
 *   src_tables    int32 [num_seqs, max_blocks_per_seq], the blocks of
 *                 context_lens[s] positions
 *   dst_tables    int32 [num_seqs, dst_blocks_per_seq], dst_blocks_per_seq *
 *                 block_size >= min(budget, the longest context)
 *   keep          int32 [num_seqs, num_kv_heads, budget]
 *   context_lens  the lengths before the eviction, each at most
 *                 max_context_len
 *   weights       fp32 or NULL, weights_stride >= max_context_len */
pkv_status_t pkv_kv_compact(
    void* k_cache, void* v_cache, float* weights, int64_t weights_stride,
    const int32_t* src_tables, int max_blocks_per_seq,
    const int32_t* dst_tables, int dst_blocks_per_seq,
    const int32_t* keep, int budget, const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
    pkv_dtype_t dtype, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * A cache held in 8 bits.
 *
 * [P2] "Why the KV cache is the thing that limits your batch": a decode step's
 * time and the pool's size are the cache's bytes.  The calls below keep K and V
 * as e4m3 codes, [num_blocks, num_kv_heads, block_size, head_dim] bytes as the
 * 16-bit caches are laid out, with one scale per row (position and KV head),
 * bfloat16 [num_blocks, num_kv_heads, block_size]:
 *   element = code * scale,  scale = 2^e,
 *   e the smallest integer >= -126 with max |element of the row| <= 448 * 2^e.
 * The division by a power of two is exact, so each element is rounded once, to
 * nearest even, and a row gives the same bits wherever it is written; read back
 * and appended again it keeps its values.  (Elements that round above their type:
 * an fp16 one from 63,488 on is held as 65,536, a bf16 one from 1.9375 2^127 on as 2^128,
 * and is infinity where it is read in that type, in an output of the attention calls,
 * too, that comes to it; appended again, its row is NaN.)  A row with a NaN or an
 * infinity is held as NaN as a whole (scale NaN, codes 0).
 *
 * The attention calls read scales as powers of two (or NaN): one of V that comes
 * from elsewhere and is none counts as the power of two below it, an infinity as NaN.
 *
 * What the attention calls hold in less than 32 bits: a query element to 2^-25 of
 * its row's largest (exactly from 2^-17 of it on in bf16, from 2^-14 on in fp16), a
 * softmax weight to 11 bits, and to 2^-31 of its row's largest weight where the V rows
 * have the same scale, 2^-24 where they have not.  So over n positions up to n 2^-31
 * (n 2^-24) of the largest weight times |v| may be lost: 2^-14 over 128k positions of
 * the same scale.  V rows may be of any sizes; what is below 2^-126 of the largest one
 * may be lost.
 *
 * pkv_block_copy copies the codes (block_bytes = num_kv_heads * block_size *
 * head_dim) and, in a call of its own, the scales (num_kv_heads * block_size *
 * 2).  Prompt chunks attend over cached blocks read back by pkv_block_read_fp8
 * (pkv_paged_attn_prefill).  Codes must be 16-byte aligned, scales 16-byte
 * aligned.
 * ---------------------------------------------------------------------- */

/* Quantise new tokens' K and V rows into their slots: pkv_kv_append for an
 * 8-bit cache, with the same slot_mapping (distinct; negative skips a token;
 * beyond the pool flags PKV_DEV_BAD_SLOT).
 *
 *   k, v          [num_tokens, num_kv_heads, head_dim] dtype, tokens *_stride
 *                 elements apart (a multiple of 8, at least a token's row)
 * Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED (head_dim or block_size not
 * built, 2^31 or more 16-element parts of rows in one call), PKV_ERR_CUDA. */
pkv_status_t pkv_kv_append_fp8(
    const void* k, int64_t k_stride, const void* v, int64_t v_stride,
    void* k_cache, void* v_cache, void* k_scales, void* v_scales,
    const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, pkv_dtype_t dtype, pkv_stream_t stream);

/* Read blocks back into 16 bits: for each pair i, block src_dst_pairs[2i] of
 * the 8-bit caches, every row of it, into block src_dst_pairs[2i + 1] of k_out
 * and v_out [num_out_blocks, num_kv_heads, block_size, head_dim].  bf16 holds
 * the products exactly (from its smallest normal number to its largest), fp16
 * rounds them once, to infinity from 65,520 on.  A source may be read into several blocks; destinations must be
 * distinct.  Ids outside the pools skip the pair and flag PKV_DEV_BAD_BLOCK_ID.
 * Errors as pkv_kv_append_fp8. */
pkv_status_t pkv_block_read_fp8(
    void* k_out, void* v_out, int num_out_blocks, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales, const int64_t* src_dst_pairs, int num_pairs,
    int num_kv_heads, int head_dim, int block_size, int num_blocks, pkv_dtype_t dtype,
    pkv_stream_t stream);

/* Norms of the query and key heads with rotary positions, in one launch: what
 * pkv_rope_kv_append does to q and k, for a cache that takes k from elsewhere,
 * with each head row first normalised,
 *   y = x * weight / sqrt(mean x^2 + eps),
 * where q_weight / k_weight is not NULL, and with a position per axis: pair i
 * is turned by positions[pair_axes[i]][t] * inv_freq[i] (a picture's tokens
 * have a height and a width, a film's a time besides).  attn_factor multiplies
 * the turned elements.  Each element is rounded once.  A token whose position
 * on axis 0 is negative is padding: nothing is written for it.
 *
 *   q_out, q, k_out, k  as q_out and q of pkv_rope_kv_append: an output may be
 *                 its input with the same stride, and must overlap neither
 *                 input otherwise
 *   q_weight, k_weight  [head_dim] dtype, or NULL
 *   eps           finite, >= 0
 *   positions     int32 [num_axes][positions_stride >= num_tokens]
 *   pair_axes     HOST array of rot_dim / 2 axis numbers below num_axes, read
 *                 before the call returns (NULL: axis 0 turns every pair)
 *   inv_freq      double [rot_dim / 2]
 * Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED (head_dim not built, 65,536
 * heads or more), PKV_ERR_CUDA. */
pkv_status_t pkv_qk_norm_rope(
    void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
    const void* q, int64_t q_stride, const void* k, int64_t k_stride,
    const void* q_weight, const void* k_weight, float eps,
    const int32_t* positions, int64_t positions_stride, int num_axes, const uint8_t* pair_axes,
    const double* inv_freq, int rot_dim, int interleaved, float attn_factor,
    int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, pkv_dtype_t dtype,
    pkv_stream_t stream);

/* pkv_paged_attn_decode over an 8-bit cache.  q and out are dtype; any group
 * size.  partition_size 0 or a multiple of 128; workspace of
 * pkv_decode_fp8_workspace_size(...) bytes.  Everything else as there. */
pkv_status_t pkv_paged_attn_decode_fp8(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* (size_t)-1 for invalid arguments or sizes the call does not support. */
size_t pkv_decode_fp8_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int max_context_len, int partition_size);

/* Attention of a tree of drafted tokens over an 8-bit cache: several guesses of
 * a sequence's next tokens are checked in one pass over its cache.
 *
 * Sequence s brings L_s = query_start[s+1] - query_start[s] <= 64 drafted
 * tokens, the last L_s positions of its context (as pkv_paged_attn_prefill;
 * their rows are already in the cache).  Query j sees every position before
 * the drafted ones, and of those the i-th where bit i of
 * tree_masks[query_start[s] + j] is set (bits from L_s on are ignored): its
 * ancestors and itself, for a tree.  A query that sees nothing gets zeros;
 * what a query does not see does not reach it, NaN included.
 *
 *   q, out        [total_queries, num_q_heads, head_dim] dtype, total_queries
 *                 >= query_start[num_seqs]; rows of out from
 *                 query_start[num_seqs] on are not written
 *   tree_masks    int64 [total_queries]
 *   max_query_len bound on L_s (at most 64; a sequence with more flags
 *                 PKV_DEV_BAD_CONTEXT_LEN, as does one whose context is
 *                 shorter than L_s)
 *   workspace     pkv_tree_fp8_workspace_size(...) bytes
 * Everything else as pkv_paged_attn_decode_fp8. */
pkv_status_t pkv_paged_attn_tree_fp8(
    void* out, const void* q, int total_queries, const int32_t* query_start, int max_query_len,
    const int64_t* tree_masks, const void* k_cache, const void* v_cache,
    const void* k_scales, const void* v_scales,
    const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len,
    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, pkv_dtype_t dtype,
    int partition_size, void* workspace, size_t workspace_bytes, pkv_stream_t stream);

/* (size_t)-1 for invalid arguments or sizes the call does not support. */
size_t pkv_tree_fp8_workspace_size(int total_queries, int max_query_len, int num_seqs,
                                   int num_q_heads, int num_kv_heads, int head_dim,
                                   int max_context_len, int partition_size);

/* Read (and optionally clear) the status word of the current device.
 * Synchronises `stream` first so that flags from work already enqueued on it
 * are visible.  flags may be NULL when only clearing. */
pkv_status_t pkv_device_status(uint32_t* flags, int clear, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Diagnostic for the kernels' bounded waits.
 *
 * Every wait inside the decode and prefill kernels (on the CTA's own copies,
 * MMA completions and warps) gives up after a limit (2 s), raises
 * PKV_DEV_WAIT_TIMEOUT in the device status word and lets the kernel end,
 * so that a wait that cannot complete never hangs the GPU.  This call
 * enqueues one such wait on a barrier that nothing completes: it returns
 * PKV_OK at once, the kernel ends after the limit, and pkv_device_status()
 * then reports PKV_DEV_WAIT_TIMEOUT.  The context stays usable.  Not part of
 * the hot path.
 * ---------------------------------------------------------------------- */
pkv_status_t pkv_debug_wait_timeout(pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Host-side refcounted block allocator (not on the device path).
 *
 * Fixed-size blocks, a block table per sequence, blocks taken only when all
 * earlier ones are full ([P2] "The page table, relocated into attention");
 * forked samples share blocks by reference count, a write into a shared,
 * partially filled block triggers copy-on-write, and blocks whose count
 * reaches zero return to the pool ([P2] "The part everyone forgets: pages
 * enable sharing, not just packing"; [P3] "Shared prefixes need ownership
 * rules").
 *
 * Policy: LIFO free list handing out 0, 1, 2, ... first; a sequence's blocks
 * are released from its last logical block to its first; copy-on-write iff
 * the write position is inside the last block and that block's count is
 * above one.  Every call that fails leaves the allocator unchanged.  The
 * allocator owns only ids and counts; the caller owns every tensor and must
 * order the device work it derives from these answers on its streams
 * ([P3] "Shared prefixes need ownership rules": a delayed device write must
 * not land in a block that has already been handed to another sequence).
 * Not thread-safe: one handle per host thread, or external locking.
 * ---------------------------------------------------------------------- */
typedef struct pkv_allocator pkv_allocator;

typedef struct {
  int64_t num_blocks;      /* pool size */
  int64_t free_blocks;     /* on the free list */
  int64_t used_blocks;     /* refcount > 0 */
  int64_t shared_blocks;   /* refcount > 1 */
  int64_t num_seqs;        /* live sequences */
  int64_t logical_tokens;  /* sum of live sequence lengths */
  int64_t filled_slots;    /* distinct physical slots holding a token */
  int64_t cow_copies;      /* copy-on-write events since creation */
} pkv_alloc_stats_t;

pkv_status_t pkv_alloc_create(int num_blocks, int block_size, pkv_allocator** out);
void pkv_alloc_destroy(pkv_allocator* a);
/* New sequence holding num_tokens >= 0 positions (ceil(n / B) blocks). */
pkv_status_t pkv_alloc_add_seq(pkv_allocator* a, int64_t seq_id, int num_tokens);
/* child shares every block of parent; both keep parent's length. */
pkv_status_t pkv_alloc_fork(pkv_allocator* a, int64_t parent, int64_t child);
/* Reserve the slot of the sequence's next token.  *cow_src / *cow_dst are
 * the block pair to copy before writing (both -1 when no copy is needed). */
pkv_status_t pkv_alloc_append_slot(pkv_allocator* a, int64_t seq_id, int64_t* slot,
                                   int64_t* cow_src, int64_t* cow_dst);
/* append_slot for n sequences in order.  slots[i] receives the slot of
 * seq_ids[i]; every copy needed is written to cow_pairs (int64 [n, 2]) and
 * *num_pairs receives their count.  All or nothing: if any sequence fails
 * (unknown id, pool exhausted) the appends already made in the batch are
 * undone, the allocator is left as before the call and *num_pairs is 0.
 * A sequence id may appear at most once per batch. */
pkv_status_t pkv_alloc_append_slots(pkv_allocator* a, const int64_t* seq_ids, int n,
                                    int64_t* slots, int64_t* cow_pairs, int* num_pairs);
/* Drop a sequence (finish or cancel); blocks reaching count 0 are freed. */
pkv_status_t pkv_alloc_free_seq(pkv_allocator* a, int64_t seq_id);
/* Shorten sequences to new_lens[i] <= their length, after an eviction.  The
 * blocks behind the new length are dropped, and a sequence that gets shorter
 * receives a fresh block in the place of every kept block that was shared when
 * the call began (another owner keeps that one; pkv_kv_compact writes every
 * row of the fresh block, so no pair to copy results).  All fresh blocks are
 * taken before any is freed, so a block the batch reads from never becomes one
 * it writes to.  All or nothing; a sequence id may appear once per batch
 * (PKV_ERR_INVALID_ARG otherwise). */
pkv_status_t pkv_alloc_shrink_seqs(pkv_allocator* a, const int64_t* seq_ids, int n,
                                   const int64_t* new_lens);
/* Host int32 rows [n, max_blocks] of physical ids, padded with -1. */
pkv_status_t pkv_alloc_block_table(pkv_allocator* a, const int64_t* seq_ids, int n,
                                   int32_t* out, int max_blocks);
/* Slots of positions [start, start + count) of a sequence (host int64). */
pkv_status_t pkv_alloc_seq_slots(pkv_allocator* a, int64_t seq_id, int start, int count,
                                 int64_t* out);
pkv_status_t pkv_alloc_seq_info(pkv_allocator* a, int64_t seq_id, int* num_tokens,
                                int* num_blocks);
pkv_status_t pkv_alloc_refcount(pkv_allocator* a, int block, int* refcount);
pkv_status_t pkv_alloc_stats(pkv_allocator* a, pkv_alloc_stats_t* out);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H_ */
