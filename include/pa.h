/*
 * pa.h -- C ABI of the GB300 (sm_103a) paged-KV-cache hot path.
 *
 * Device operations and a host block manager:
 *   pa_kv_write     scatter new tokens' K/V into physical cache blocks through slot_mapping
 *   pa_attention    paged decode and chunked-prefill attention through block_table
 *   pa_write_attention  the two above in one call (the write fused into decode)
 *   pa_kv_write_fp8 / pa_attention_fp8  the same over FP8 (E4M3) caches
 *   pa_attention_grouped  decode attention reading a shared prefix once per group
 *   pa_copy_blocks  copy whole physical blocks (the copy step of copy-on-write)
 *   pa_swap_blocks  move whole blocks between the GPU pool and a CPU pool (preemption)
 *   pa_advance_batch    a step's block tables, slots and positions from request lengths, on the GPU
 *   pa_norm_rope_write  RMS norm and rotary positions of query and key heads, and the cache write
 *   pa_block_bounds / pa_block_scores / pa_select_blocks / pa_attention_sparse
 *                   attention over the blocks that a cheap score selects for each query token
 *   pa_kv_write_int / pa_kv_read_int / pa_attention_int
 *                   caches of 4- or 8-bit integer codes: quantised as written, read back, attended
 *   pa_attention_packed  causal attention of whole prompts over packed rows (no pages)
 *   pa_bm_*         host-side block accounting: free queue, block tables, ref counts, CoW
 *
 * Conventions shared by every entry point:
 *  - Cache layout: k_cache and v_cache are each [num_blocks, block_size, num_kv_heads,
 *    head_dim], row-major and contiguous, element type `dtype`. A "slot" is one token
 *    position in the pool: slot = block * block_size + offset, i.e. the row index of
 *    the cache viewed as [num_blocks * block_size, num_kv_heads * head_dim].
 *  - Pointers marked "device" must point to device memory of the current CUDA device,
 *    owned by the caller and 16-byte aligned; the library never allocates, frees or
 *    synchronises (except pa_read_device_errors, which synchronises by design). Work is
 *    enqueued on `stream` (0 = legacy default stream) and the call returns before it runs.
 *  - Return value: a pa_status. Argument checks happen before anything is launched; a
 *    call that returns an error has enqueued nothing. PA_ERR_CUDA means a launch
 *    failed; pa_last_cuda_error() gives the cudaError_t of the calling thread's last one.
 *  - Index values inside device arrays (slots, block ids, lengths) cannot be checked on
 *    the host. Kernels check them against the sizes passed in and skip any access that
 *    would leave the buffers; such a skip sets a bit in a per-device error word that
 *    pa_read_device_errors() returns. Results are then unspecified but no memory outside
 *    the arguments is touched.
 *  - Per-device state: the library looks up a few device addresses (the error word, the
 *    fixed scratch of pa_attention_fixed_scratch) and creates a side stream with two
 *    events once per device, on first use, and keeps them until exit. A process that
 *    resets a device (cudaDeviceReset) or otherwise destroys its primary context must not
 *    call the library for that device afterwards: the kept addresses and handles would be
 *    stale.
 *
 * Sources (the pages this library restates):
 *  [docs]  "vLLM", docs.acceleratez.fun/llm/model-inference/vllm.html -- PagedAttention
 *          (blocks, block table, algorithm flow), memory-utilisation arithmetic,
 *          Copy-on-Write (reference counting, copy before a divergent write).
 *  [flow]  vLLM 0.10.0 flow analysis, ascendai.csdn.net/69ac14cf54b52172bc5fa372.html --
 *          3.2 Scheduler (prefill compute-bound, decode memory-bound, chunked prefill
 *          mixed with decodes), 3.3 KV Manager (slot, block, pool, slot_mapping),
 *          3.5 Attention (q is the flattened token batch; metadata block_table,
 *          slot_mapping, query_start_loc).
 *  [read]  vLLM code reading, sourceaix.com/community/post/7301643446391930880 --
 *          5.1.1 single request (logical vs physical blocks, '# filled'),
 *          5.2.1 parallel sampling (shared blocks, ref count, copy-on-write).
 *  [intro] VLLM overview, dn008.com.cn/news/553482 -- 2.1 KV cache (causal mask); 4
 *          scheduler (waiting / running / swapped queues, swap phase).
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* pa_stream_t;

typedef enum { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2 /* caches only: see pa_kv_write_fp8 */ } pa_dtype;

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, misaligned pointer, bad shape */
  PA_ERR_UNSUPPORTED = 2,  /* a valid shape the library has no kernel for */
  PA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than pa_attention_workspace_size */
  PA_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  PA_ERR_NO_BLOCKS = 5,    /* block manager: not enough free blocks now */
  PA_ERR_TOO_LARGE = 6,    /* block manager: the sequence can never fit the pool */
  PA_ERR_NOT_FOUND = 7,    /* block manager: unknown sequence id, or id already in use */
} pa_status;

/* Bits of the per-device error word (see pa_read_device_errors). */
#define PA_DEVERR_SLOT_RANGE   0x1u  /* a slot >= num_blocks * block_size was skipped */
#define PA_DEVERR_BLOCK_RANGE  0x2u  /* a block id outside [0, num_blocks) was skipped */
#define PA_DEVERR_SEQ_RANGE    0x4u  /* seq_len > max_blocks_per_seq * block_size, q_len > seq_len, or more
                                        queries or tokens than the call announced */
#define PA_DEVERR_TIMEOUT      0x8u  /* a pipeline wait gave up (the kernel returned early) */
#define PA_DEVERR_SLOT_MISMATCH 0x10u /* pa_write_attention: a decode token's slot is not its position's slot */
#define PA_DEVERR_NO_BLOCKS    0x20u  /* pa_advance_batch: the free list does not hold the blocks of the step */
#define PA_DEVERR_POSITION     0x40u  /* pa_norm_rope_write: a position outside [0, max_position) */

const char* pa_status_string(int status);
int pa_last_cuda_error(void);

/* Reads the current device's error word (synchronising the device) and clears it if
 * `clear` is non-zero. Returns PA_OK or PA_ERR_CUDA. */
int pa_read_device_errors(unsigned int* flags_out, int clear);

/* ------------------------------------------------------------------------------
 * pa_kv_write -- [docs] PagedAttention, algorithm flow (prefill step c, decode step d:
 * store each new token's KV in its physical block); [flow] 3.3 KV Manager (the model
 * runner builds slot_mapping; attention finds each token's KV through it).
 *
 * For every t in [0, num_tokens) with s = slot_mapping[t] >= 0:
 *     k_cache[s / block_size, s % block_size, :, :] = k[t, :, :]   (same for v)
 * A negative slot marks a padding token: nothing is written for it.
 *
 * k, v          device, [num_tokens, num_kv_heads, head_dim], contiguous, `dtype`
 * k_cache, ...  device, cache layout above (written in place)
 * slot_mapping  device, int64 [num_tokens]; slots must be distinct (no two tokens
 *               written to one slot in a call -- which one would win is unspecified)
 * num_tokens    >= 0 (0 enqueues nothing)
 * Byte-exact copy; no arithmetic on the values.
 * --------------------------------------------------------------------------- */
int pa_kv_write(const void* k, const void* v, void* k_cache, void* v_cache,
                const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                int block_size, int num_kv_heads, int head_dim, pa_dtype dtype,
                pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_copy_blocks -- [docs] Copy-on-Write (copy the old block's content into the newly
 * allocated block before the divergent write); [read] 5.2.1 (A1's block 1 copied to 3).
 *
 * For each i in [0, num_pairs): src = block_mapping[2i], dst = block_mapping[2i+1]:
 *     k_cache[dst] = k_cache[src]; v_cache[dst] = v_cache[src]   (all block_size slots)
 * block_mapping  device, int64 [num_pairs, 2]
 * Pairs are applied concurrently: no dst may repeat or appear as another pair's src
 * (pairs emitted by the block manager below always satisfy this: every dst is a block
 * just taken from the free queue and every src is a block still held by others).
 * Byte-exact copy.
 * --------------------------------------------------------------------------- */
int pa_copy_blocks(void* k_cache, void* v_cache, const int64_t* block_mapping,
                   int64_t num_pairs, int64_t num_blocks, int block_size, int num_kv_heads,
                   int head_dim, pa_dtype dtype, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_attention -- [flow] 3.5 Attention (q = flattened tokens of the batch, requests
 * delimited by query_start_loc; K/V read from the whole cache through block_table);
 * [docs] PagedAttention (block table: logical block -> physical block); [read] 5.1.1
 * (attention runs over the logical blocks, as if contiguous); [intro] 2.1 (causal);
 * [flow] 3.2 (chunked prefill mixed with decodes in one batch).
 *
 * For request s with q_len = query_start_loc[s+1] - query_start_loc[s] and
 * L = seq_lens[s] (keys, including the request's new tokens), query row j (token
 * t = query_start_loc[s] + j) sits at position p = L - q_len + j and, for each query
 * head h with KV head g = h / (num_heads / num_kv_heads):
 *     K_i = k_cache[block_table[s, i / block_size], i % block_size, g, :]   (V alike)
 *     out[t, h, :] = sum_{i<=p} softmax_i(scale * <q[t, h, :], K_i>) * V_i
 * Softmax and accumulation in fp32; out is written in `dtype` (bf16 rounded to nearest
 * even). Requests with q_len == 1 run the split-K decode kernel; q_len >= 2 the prefill
 * kernel; q_len == 0 produces no rows. Requires q_len <= L.
 * With rows of both kinds (max_query_len >= 2) and the tensor-core kernels for both (see
 * "Prefill kernels" below; block size 8, 16, 32, 64 or 128) the two kernels run side by
 * side: the call forks an internal stream of the highest priority off `stream` (event
 * record and wait), runs the decode kernels there on 3/5 of the SMs (1/2 with E4M3
 * caches) and joins it back before returning -- also when a launch fails after the fork --
 * so later work on `stream` is ordered after the whole call, as for one stream. The first such call
 * on a device creates that stream and two events (kept until exit). While `stream` is
 * being captured into a CUDA graph the call keeps every kernel on `stream` instead (the
 * internal stream is shared by all callers of the device and must not join a capture).
 * The decode rows' bits differ between the two ways (a split over fewer CTAs beside the
 * prefill kernel; same tolerance).
 * Prefill kernels: the tensor-core kernel takes bf16 q and out over bf16 caches (head_dim
 * 64 / 128) or E4M3 caches (head_dim 128; see pa_attention_fp8), at most 4096 requests,
 * block size 8, 16, 32, 64 or 128; other prefill batches (fp32, block sizes 1, 2, 4 or
 * above 128, more than 4096 requests) run a CUDA-core kernel with the same result within
 * the tolerance, many times slower.
 * The result does not depend on which physical blocks hold the tokens: the reduction
 * order is fixed by positions only, so relabelling block ids gives identical bits.
 *
 * out           device, [num_tokens, num_heads, head_dim], `dtype` (written, never read);
 *               may also be page-locked host memory mapped into the unified address
 *               space: the kernels then store the rows over the CPU-GPU link and the host
 *               sees them once the stream has been synchronised
 * q             device, [num_tokens, num_heads, head_dim], `dtype`; for a decode-only
 *               batch (max_query_len <= 1) on the tensor-core decode kernel it may also be
 *               page-locked host memory mapped into the unified address space: the kernel
 *               then reads the rows over the CPU-GPU link (plain loads, no copy). q is
 *               checked with cudaPointerGetAttributes: pageable host memory or another
 *               device's memory gives PA_ERR_INVALID_ARG; host memory with prefill rows gives
 *               PA_ERR_INVALID_ARG, and on a shape the tensor-core decode kernel does not take
 *               PA_ERR_UNSUPPORTED (all before anything is enqueued)
 * block_table   device, int32 [num_seqs, max_blocks_per_seq] (entries past a request's
 *               ceil(L / block_size) blocks are never read)
 * seq_lens      device, int32 [num_seqs]
 * query_start_loc device, int32 [num_seqs + 1], non-decreasing, [0] = 0, [num_seqs] =
 *               num_tokens
 * max_query_len host: an upper bound of every q_len (sizes the prefill grid)
 * max_seq_len   host: an upper bound of every L (validated against the table width)
 * workspace     device scratch of at least pa_attention_workspace_size() bytes (at least
 *               16: its last part holds the prefill kernel's work counter, which the call
 *               zeroes on its stream before that kernel); no initial contents needed; must
 *               not be used by another call that may run concurrently.
 * Supported: dtype PA_F32 / PA_BF16; head_dim 64 / 128; num_heads / num_kv_heads in
 * {1, 2, 4, 8}; block_size a divisor of 16 (1, 2, 4, 8, 16) or a multiple of 16.
 * --------------------------------------------------------------------------- */
int pa_attention_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                int head_dim, size_t* bytes_out);

int pa_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                 const int32_t* query_start_loc, int num_seqs, int num_tokens,
                 int max_query_len, int max_seq_len, int num_heads, int num_kv_heads,
                 int head_dim, int block_size, int64_t num_blocks, float scale,
                 pa_dtype dtype, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_write_attention -- pa_kv_write followed by pa_attention, in one call:
 * [docs] PagedAttention algorithm flow (decode step d stores the new token's KV in its
 * block, then attends over all of the request's blocks); [flow] 3.3 / 3.5 (slot_mapping
 * feeds the cache write that precedes attention in the same forward pass).
 *
 * Result (cache and out) identical to pa_kv_write(k_new, v_new, ..., slot_mapping,
 * num_tokens, ...) then pa_attention(...) on one stream, under one extra contract: for
 * a request with q_len == 1 at length L, slot_mapping of its token is the slot of
 * position L - 1, block_table[s, (L-1) / block_size] * block_size + (L-1) % block_size
 * (or negative: a padding token, nothing written). A token breaking this sets
 * PA_DEVERR_SLOT_MISMATCH; its KV is still written, its request's output is then
 * unspecified.
 *  - max_query_len <= 1 (a decode-only batch): one launch pair. The split-K CTA that
 *    streams a request's last 16 positions for a KV-head group first copies that group's
 *    slice of the new K/V row into the cache, then reads it back with the rest, so the
 *    new token costs one write and no separate kernel.
 *  - max_query_len >= 2: the cache write is a separate kernel ahead of the attention
 *    kernels (prefill rows read their new tokens through many CTAs).
 * k_new, v_new  device, [num_tokens, num_kv_heads, head_dim], `dtype`, 16-byte aligned;
 *               like q, page-locked host memory for decode-only batches (read over the link)
 * slot_mapping  device, int64 [num_tokens], distinct non-negative slots
 * Other arguments, validation, workspace and errors as pa_kv_write and pa_attention;
 * validation happens before anything is enqueued.
 * --------------------------------------------------------------------------- */
int pa_write_attention(void* out, const void* q, const void* k_new, const void* v_new,
                       const int64_t* slot_mapping, void* k_cache, void* v_cache,
                       const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                       const int32_t* query_start_loc, int num_seqs, int num_tokens,
                       int max_query_len, int max_seq_len, int num_heads, int num_kv_heads,
                       int head_dim, int block_size, int64_t num_blocks, float scale,
                       pa_dtype dtype, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_attention_grouped -- pa_attention for a decode batch (one query per request) whose
 * requests come in groups sharing a prefix of physical blocks: [read] 5.2.1 (samples of one
 * prompt share its blocks), [docs] Copy-on-Write (shared blocks, reference counts).
 *
 * Same result as pa_attention. The grouping only changes how the work is done: for group
 * g the first shared_len[g] positions are read once and multiplied against the queries of
 * all its members together (the members' query heads become one set of matrix rows), and
 * each member's remaining positions run on their own; the pieces are merged per request.
 *  seq_group     device int32 [num_seqs]: the request's group, or -1
 *  group_range   device int32 [num_groups, 2]: group g's members are the consecutive
 *                requests [group_range[2g], group_range[2g+1])
 *  shared_len    device int32 [num_groups]: positions [0, shared_len[g]) of every member
 *                are the same physical slots (same block ids in their tables); the library
 *                reads them through the first member's table
 * The kernel uses whole 16-token chunks below shared_len and every member's length, and
 * runs a group ungrouped when members x (num_heads / num_kv_heads) > 16 or it has fewer
 * than 2 members; a request whose seq_group does not match group_range runs ungrouped.
 * bf16 only (q, out, caches); head_dim 64 / 128; block size 8 or a multiple of 16;
 * num_heads / num_kv_heads <= 8. Workspace from pa_attention_grouped_workspace_size.
 * pa_bm_batch_groups builds the three arrays from the block manager's tables.
 * --------------------------------------------------------------------------- */
int pa_attention_grouped_workspace_size(int num_seqs, int num_groups, int num_heads, int num_kv_heads,
                                        int head_dim, size_t* bytes_out);

int pa_attention_grouped(void* out, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* query_start_loc, int num_seqs, int num_tokens, int max_seq_len,
                         int num_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                         float scale, pa_dtype dtype, const int32_t* seq_group, const int32_t* group_range,
                         const int32_t* shared_len, int num_groups, void* workspace, size_t workspace_bytes,
                         pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * FP8 KV cache -- [docs] quantisation support (FP8: 8-bit, 2x smaller than 16-bit storage).
 *
 * k_cache / v_cache hold one E4M3 code per element (PA_FP8_E4M3: 1 sign bit, 4 exponent
 * bits with bias 7, 3 mantissa bits, no infinities, largest finite 448), same layout as
 * above with 1-byte elements. A code c of the K (V) cache stands for value(c) * k_scale
 * (v_scale): one positive scale per cache, chosen by the caller (e.g. max |K| / 448).
 *
 * pa_kv_write_fp8: for every t with s = slot_mapping[t] >= 0,
 *     k_cache[s / B, s % B, :, :] = E4M3(k[t, :, :] / k_scale)      (same for v)
 * where x is widened to binary32, divided once (binary32, round to nearest even), then
 * rounded to E4M3 (nearest, ties to even; magnitudes beyond 448 saturate to 448).
 * k, v are [num_tokens, num_kv_heads, head_dim] in `in_dtype` (PA_BF16 or PA_F32).
 * num_kv_heads * head_dim must be a multiple of 16. Other rules as pa_kv_write.
 *
 * pa_attention_fp8: pa_attention over E4M3 caches with bf16 q and out: K and V are
 * read as value(code) * scale (exact in fp32 up to the scale product), the rest is
 * pa_attention's arithmetic. The split-K decode kernel reads the 1-byte cache directly
 * (half the bytes of bf16). Requests with q_len >= 2 run the tensor-core prefill kernel
 * when head_dim is 128 and the block size is 8, 16, 32, 64 or 128 (at most 4096 requests):
 * it converts each K/V tile of codes to f16 in shared memory (exact) and the pair's queries
 * from bf16 to f16, so q must lie within f16's range (|q| < 65520; magnitudes below 2^-24
 * become 0) and P is rounded to f16; other prefill shapes run the CUDA-core kernel.
 * Workspace from pa_attention_workspace_size. pa_copy_blocks takes PA_FP8_E4M3 caches
 * (byte copy), and pa_kv_write with dtype PA_FP8_E4M3 copies already-encoded rows.
 * --------------------------------------------------------------------------- */
int pa_kv_write_fp8(const void* k, const void* v, pa_dtype in_dtype, void* k_cache, void* v_cache,
                    const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks, int block_size,
                    int num_kv_heads, int head_dim, float k_scale, float v_scale, pa_stream_t stream);

int pa_attention_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                     const int32_t* query_start_loc, int num_seqs, int num_tokens, int max_query_len,
                     int max_seq_len, int num_heads, int num_kv_heads, int head_dim, int block_size,
                     int64_t num_blocks, float scale, float k_scale, float v_scale, void* workspace,
                     size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_swap_blocks -- [read] 6.2.1 (a preempted sequence group's KV blocks are swapped out
 * to the CPU, and swapped back in when GPU resources return); [intro] 4, scheduling flow,
 * swap phase (the swapped queue lives in CPU memory).
 *
 * For each i in [0, num_pairs): s = block_mapping[2i], d = block_mapping[2i+1]:
 *     dst_k[d] = src_k[s]; dst_v[d] = src_v[s]     (whole blocks, byte copy)
 * src_* pools have src_num_blocks blocks, dst_* pools dst_num_blocks, all with the block
 * geometry [block_size, num_kv_heads, head_dim] of `dtype` (PA_F32 / PA_BF16 /
 * PA_FP8_E4M3). Each pool may be device memory or pinned host memory (cudaHostAlloc or
 * cudaHostRegister'ed, used through its unified address): the kernel moves the blocks
 * over the CPU-GPU link itself, one launch per call. block_mapping: int64 [num_pairs, 2],
 * device or pinned host memory. No dst may repeat. Out-of-range ids are skipped and set
 * PA_DEVERR_BLOCK_RANGE. The pairs come from pa_bm_swap_out / pa_bm_swap_in. Every
 * pointer is checked with cudaPointerGetAttributes before the launch: another device's
 * memory, pageable host memory or host memory not mapped at its own address gives
 * PA_ERR_INVALID_ARG.
 * --------------------------------------------------------------------------- */
int pa_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v,
                   const int64_t* block_mapping, int64_t num_pairs, int64_t src_num_blocks,
                   int64_t dst_num_blocks, int block_size, int num_kv_heads, int head_dim,
                   pa_dtype dtype, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_advance_batch -- the metadata of a step, from request lengths, on the device: [flow]
 * 3.3 KV Manager and 3.5 Attention (block_table, slot_mapping, query_start_loc); [docs]
 * PagedAttention, algorithm flow (a token that must go into a full block takes a new one);
 * [read] 5.1.1 (ceil(n / B) blocks hold n tokens).
 *
 * Request s holds c = seq_lens[s] tokens in the first ceil(c / B) entries of its table row and
 * gets n = query_lens[s] >= 0 new ones. In request order it takes the next
 * ceil((c + n) / B) - ceil(c / B) blocks of the free list -- what the host block manager
 * takes for the same appends with its free queue in the same order -- and
 *     block_table[s, ceil(c / B) + i] = its i-th new block
 *     query_start_loc[s + 1] = n_0 + ... + n_s,  query_start_loc[0] = 0
 *     seq_lens_out[s] = c + n
 *     for token t = query_start_loc[s] + j, p = c + j:
 *         positions[t] = p,  slot_mapping[t] = block_table[s, p / B] * B + p % B
 *     free_head_out = free_head + the blocks taken
 * Tokens behind the last request's (up to num_tokens) get slot -1 (padding: nothing is
 * written for them) and position 0. Nothing here knows about shared blocks: a request whose
 * last, partly filled block is shared must have been given its copy first (pa_copy_blocks).
 *
 * A step that cannot be built changes neither table nor lengths: with a negative length, more
 * than num_tokens new tokens, or a request longer than its table row (PA_DEVERR_SEQ_RANGE), or
 * too few blocks in the free list (PA_DEVERR_NO_BLOCKS), query_start_loc is all 0, every slot
 * -1, seq_lens_out = seq_lens and free_head_out = free_head. A block id outside
 * [0, num_blocks) gives its tokens slot -1 (PA_DEVERR_BLOCK_RANGE).
 *
 * block_table   device, int32 [num_seqs, max_blocks_per_seq]; only the new entries are written
 * seq_lens, query_lens  device, int32 [num_seqs]
 * free_blocks   device, int32 [num_free]; free_head: device, int32 [1], entries already taken
 * seq_lens_out, free_head_out  device; each may be its input array (a captured graph can then be
 *               replayed step after step), else must not overlap any input
 * query_start_loc  device, int32 [num_seqs + 1]; slot_mapping: device, int64 [num_tokens];
 *               positions: device, int32 [num_tokens]
 * num_tokens    entries of slot_mapping and positions: at least the new tokens of the step
 * num_seqs and num_tokens may be 0 (num_seqs = 0: padding only). One launch, no workspace.
 * --------------------------------------------------------------------------- */
int pa_advance_batch(int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                     const int32_t* query_lens, const int32_t* free_blocks, int num_free,
                     const int32_t* free_head, int32_t* seq_lens_out, int32_t* free_head_out,
                     int32_t* query_start_loc, int64_t* slot_mapping, int32_t* positions,
                     int num_seqs, int num_tokens, int block_size, int64_t num_blocks,
                     pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_norm_rope_write -- the rows a projection made, turned into queries and cached keys and
 * values in one pass: [docs] PagedAttention, algorithm flow (store each new token's KV in its
 * physical block); [flow] 3.5 (positions and slot_mapping of the flattened token batch). The
 * norm and the rotation have no counterpart in the pages.
 *
 * For every token t, and every head row x of q[t] and k[t] (head_dim elements):
 *     y = x / sqrt(mean(x^2) + eps) * weight          (q_weight / k_weight; null: y = x)
 *     for each pair i in [0, rot_dim / 2), elements (a, b) = (i, i + rot_dim / 2), or
 *     (2 i, 2 i + 1) when `interleaved`:
 *         y'_a = y_a cos - y_b sin,  y'_b = y_b cos + y_a sin
 *         cos = cos_sin[p, i], sin = cos_sin[p, rot_dim / 2 + i], p = the position of i's axis
 *     (elements from rot_dim on keep y), then q_out[t] = y' of q, and with slot = slot_mapping[t]
 *     >= 0: k_cache[slot] = y' of k, v_cache[slot] = v[t] (negative: nothing is cached).
 * Arithmetic in fp32, rounded once, to the output's type; E4M3 caches store
 * E4M3(x / k_scale) (v_scale) as pa_kv_write_fp8 does.
 *
 * q, k, v       device, `dtype` (PA_BF16 / PA_F32): token t's heads are contiguous at
 *               q + t * q_stride elements (k_stride, v_stride alike), so all three may be slices
 *               of one projection's output. Strides are multiples of 16 bytes and at least the
 *               row; pointers are 16-byte aligned.
 * q_out         device, [num_tokens, num_heads, head_dim], `dtype`, contiguous; may be q itself
 *               when q is contiguous, else must not overlap the inputs
 * q_weight, k_weight  device, [head_dim], `dtype`, or null
 * cos_sin       device, fp32 [max_position, rot_dim]: the cosines of a position's rot_dim / 2
 *               angles, then their sines
 * positions     device, int32 [num_axes, num_tokens]. A token with a position outside
 *               [0, max_position) is skipped: its q_out row and cache slot stay as they are
 *               (PA_DEVERR_POSITION)
 * num_axes      1 to 4; sections: host, [num_axes] pair counts that sum to rot_dim / 2: axis 0
 *               turns the first sections[0] pairs, and so on (null with one axis). E.g. time,
 *               height and width of an image's tokens
 * slot_mapping  device, int64 [num_tokens], distinct non-negative slots
 * cache_dtype   `dtype`, or PA_FP8_E4M3; caches as everywhere
 * Supported: head_dim 64 / 128, rot_dim a multiple of 16 up to head_dim.
 * --------------------------------------------------------------------------- */
int pa_norm_rope_write(void* q_out, const void* q, const void* k, const void* v, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, const void* q_weight, const void* k_weight,
                       float eps, const float* cos_sin, int max_position, int rot_dim, int interleaved,
                       const int32_t* positions, int num_axes, const int* sections,
                       const int64_t* slot_mapping, void* k_cache, void* v_cache, int64_t num_tokens,
                       int64_t num_blocks, int block_size, int num_heads, int num_kv_heads,
                       int head_dim, pa_dtype dtype, pa_dtype cache_dtype, float k_scale,
                       float v_scale, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * Block-sparse attention: each query token attends only to the blocks that a cheap score
 * selects for it. No counterpart in the pages; built on their blocks and tables ([docs]
 * PagedAttention, [flow] 3.5). A step runs
 *     pa_block_bounds -> pa_block_scores -> pa_select_blocks -> pa_attention_sparse
 * on one stream after the cache write, over the same batch arguments as pa_attention
 * (block_table, seq_lens, query_start_loc: token t of request s sits at position
 * p = seq_lens[s] - q_len + t - query_start_loc[s]; its context is blocks 0 .. p / block_size).
 * Rows of tokens that belong to no request (behind the last one) are left as they are. A request
 * with q_len > seq_len, or longer than its table row, sets PA_DEVERR_SEQ_RANGE and its rows are
 * left as they are; so may one of more than max_query_len queries.
 * Supported: head_dim 64 / 128; num_heads / num_kv_heads in {1, 2, 4, 8}; block_size a multiple
 * of 16; bf16 queries over bf16 or E4M3 caches (any of them for bounds, scores and selection,
 * which never read the queries' cache). No workspace; every kernel on `stream`.
 *
 * pa_block_bounds: for every block that holds one of the request's new tokens (positions
 * seq_lens - q_len .. seq_lens - 1), id = its physical block:
 *     bounds[id, g, 0, :] = min_i K_i[g, :],  bounds[id, g, 1, :] = max_i K_i[g, :]
 * over the block's positions below seq_lens, recomputed from the cache (E4M3: the codes'
 * values, without k_scale). Exact. bounds: device, bf16 [num_blocks, num_kv_heads, 2, head_dim],
 * kept beside the cache by the caller. Blocks that came to hold keys in another way (copied,
 * swapped in, cached prefixes of another pool) get their bounds by a call whose
 * query_start_loc covers their positions. Two requests that share a block must agree on its
 * keys (shared blocks are full, or hold the same tokens). num_tokens: query_start_loc[num_seqs]
 * or more (it sizes the grid when max_query_len > 1; a batch with more tokens then sets
 * PA_DEVERR_SEQ_RANGE, and some of its blocks keep their old bounds).
 *
 * pa_block_scores: for block b of token t's context and KV head g
 *     scores[t, g, b] = max_h sum_d max(q_hd lo_d, q_hd hi_d)      (h: the group's query heads)
 * -- no logit of the block, before the softmax scale (and k_scale), is larger -- and -inf for
 * the blocks behind the context. scores: device, fp32 [num_tokens, num_kv_heads, score_width],
 * score_width >= ceil(max_seq_len / block_size). A block id outside [0, num_blocks) scores
 * -inf (PA_DEVERR_BLOCK_RANGE). Bounds and queries are taken as finite: a NaN or infinite one
 * gives scores of no meaning, never an access out of range.
 *
 * pa_select_blocks: block_idx[t, g, :] = the token's blocks in ascending order: the first
 * `init_blocks` and the last `local_blocks` blocks of its context always, the others by the
 * largest score, equal scores by the lowest block, never one of score -inf or NaN; entries
 * behind them are -1. block_idx: device, int32 [num_tokens, num_kv_heads, num_select],
 * init_blocks + local_blocks <= num_select.
 *
 * pa_attention_sparse: with the blocks listed in block_idx[t, g, :] (entries below 0 are
 * skipped, in any order; a block listed twice counts twice, one behind the context not at all):
 *     out[t, h, :] = sum_i softmax_i(scale <q[t, h, :], K_i>) V_i
 * over their positions i <= p; zeros where there is none. Keys past the request's length are
 * never read. K and V are value(code) * k_scale (v_scale) for E4M3 caches, as in
 * pa_attention_fp8 (with its range of q); k_scale and v_scale are 1 for bf16 caches. An entry
 * >= max_blocks_per_seq or a block id outside [0, num_blocks) is skipped
 * (PA_DEVERR_BLOCK_RANGE). out, q: device, bf16 [num_tokens, num_heads, head_dim]. The result
 * does not depend on which physical blocks hold the tokens, nor on what else runs.
 * --------------------------------------------------------------------------- */
int pa_block_bounds(void* bounds, const void* k_cache, const int32_t* block_table, int max_blocks_per_seq,
                    const int32_t* seq_lens, const int32_t* query_start_loc, int num_seqs,
                    int num_tokens, int max_query_len, int max_seq_len, int num_kv_heads,
                    int head_dim, int block_size, int64_t num_blocks, pa_dtype cache_dtype,
                    pa_stream_t stream);

int pa_block_scores(float* scores, int score_width, const void* q, const void* bounds,
                    const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                    const int32_t* query_start_loc, int num_seqs, int num_tokens, int max_query_len,
                    int max_seq_len, int num_heads, int num_kv_heads, int head_dim, int block_size,
                    int64_t num_blocks, pa_stream_t stream);

int pa_select_blocks(int32_t* block_idx, int num_select, const float* scores, int score_width,
                     const int32_t* seq_lens, const int32_t* query_start_loc, int num_seqs,
                     int num_tokens, int num_kv_heads, int block_size, int init_blocks,
                     int local_blocks, pa_stream_t stream);

int pa_attention_sparse(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                        const int32_t* query_start_loc, const int32_t* block_idx, int num_select,
                        int num_seqs, int num_tokens, int max_seq_len, int num_heads,
                        int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                        float scale, pa_dtype cache_dtype, float k_scale, float v_scale,
                        pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * Integer-coded caches: keys and values held as 4- or 8-bit codes with a smallest value and a step
 * for every token and KV head, so that a cache of head_dim 128 takes 68 (132) bytes a row instead of
 * bf16's 256, and no scale has to be known before the rows are. No counterpart in the pages beyond
 * their blocks, slots and tables ([docs] PagedAttention, [flow] 3.3, 3.5). A serving loop runs
 *   prompt   pa_kv_write_int; pa_attention_packed over the prompt's own rows
 *   chunk    pa_kv_write_int; pa_kv_read_int of the context ahead of the chunk's rows, then
 *            pa_attention_packed over both
 *   decode   pa_kv_write_int; pa_attention_int
 *
 * Row x (head_dim elements, one token and KV head), with N = 2^bits - 1, in binary32:
 *     lo   = the largest bfloat16 not above min(x)
 *     step = max(2^-126, the smallest bfloat16 not below (max(x) - lo) / N)
 *     code = rint((x - lo) inv), ties to even, inv = 1 / step (the product not rounded before rint)
 * and a code stands for lo + step code. The error of an element is at most half a step. A row that
 * holds a NaN or an infinity, or whose spread passes the largest float, reads back as NaN.
 *
 * k_cache, v_cache: device, uint8 [num_blocks, num_kv_heads, block_size * (head_dim * bits / 8 + 4)]:
 * of each block and head first the rows' codes (token after token; element 2 i in the low half of
 * byte i when bits = 4), then a row's lo and step, both bfloat16, token after token. A block's bytes lie
 * together: pa_copy_blocks and pa_swap_blocks move them as caches of PA_FP8_E4M3 with one "head" of
 * block_size * (head_dim * bits / 8 + 4) "elements" and num_kv_heads "tokens" a block.
 * Supported: head_dim 64 / 128; block_size a multiple of 4; bits 4 / 8; else PA_ERR_UNSUPPORTED.
 * Every kernel on `stream`.
 *
 * pa_kv_write_int: for every t with slot = slot_mapping[t] >= 0 the rows of k[t] and v[t] become the
 * codes of that slot; negative slots are padding. k, v: device, `dtype` (PA_BF16 / PA_F32), token t's
 * heads contiguous at k + t * k_stride elements (v_stride alike; strides multiples of 16 bytes and at
 * least the row). slot_mapping: device, int64 [num_tokens], distinct non-negative slots; one outside
 * the cache is skipped (PA_DEVERR_SLOT_RANGE).
 *
 * pa_kv_read_int: for request s and i in [0, seq_lens[s] - start_pos[s]), the values of position
 * start_pos[s] + i go to row row_start_loc[s] + i of k_out and v_out (device, [num_rows, num_kv_heads,
 * head_dim], `dtype` PA_BF16 / PA_F32, computed in fp32 and rounded once). start_pos: device, int32
 * [num_seqs], or null (all 0). row_start_loc: device, int32 [num_seqs + 1], not decreasing. Rows of a
 * request behind those (room for a chunk's own rows) and rows of no request are left as they are. A request
 * whose positions do not fit its rows (those below num_rows; it may have none) or its table, or a
 * negative one, sets PA_DEVERR_SEQ_RANGE; a block id outside [0, num_blocks) PA_DEVERR_BLOCK_RANGE;
 * their rows are left as they are. With num_rows = 0 nothing is launched, and so nothing reported.
 *
 * pa_attention_int: pa_attention over such caches, q and out bf16 [num_tokens, num_heads, head_dim]:
 * token j of a request's q_len sits at position seq_lens - q_len + j and sees the positions up to its
 * own. Made for decode and a few drafted tokens: 8 of a request's (token, query head) rows of a KV head
 * share one pass over its codes, 16 where max_query_len tokens make more than 8 (any num_heads that
 * num_kv_heads divides); a long chunk is faster through pa_kv_read_int and pa_attention_packed. Rows of no
 * request are left as they are; a request with more than max_query_len queries, more keys than max_seq_len,
 * or q_len > seq_len sets PA_DEVERR_SEQ_RANGE and its rows are left as they are (other requests' too, where
 * query_start_loc decreases). The positions of a block id outside [0, num_blocks) are skipped
 * (PA_DEVERR_BLOCK_RANGE); a token that sees no others gets zeros. A key or value row that reads back as
 * NaN gives NaN to the tokens that see it, and to no other. Logits are fp32, with their own range and
 * that of scale sum_d |q_d| 2^bits; so are the sums over the keys before the division, finite for values
 * below 2^119 / seq_len. workspace: device, pa_attention_int_workspace_size bytes, 16-byte
 * aligned, no contents needed; calls that may overlap on the GPU need one each. The result depends on
 * nothing but the arguments' contents and the GPU's number of SMs. num_seqs <= 4096
 * (PA_ERR_UNSUPPORTED).
 * --------------------------------------------------------------------------- */
int pa_kv_write_int(const void* k, const void* v, int64_t k_stride, int64_t v_stride, pa_dtype dtype,
                    void* k_cache, void* v_cache, const int64_t* slot_mapping, int64_t num_tokens,
                    int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, int bits,
                    pa_stream_t stream);

int pa_kv_read_int(void* k_out, void* v_out, pa_dtype dtype, const void* k_cache, const void* v_cache,
                   const int32_t* block_table, int max_blocks_per_seq, const int32_t* start_pos,
                   const int32_t* seq_lens, const int32_t* row_start_loc, int num_seqs, int64_t num_rows,
                   int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, int bits,
                   pa_stream_t stream);

int pa_attention_int_workspace_size(int num_seqs, int num_tokens, int num_heads, int num_kv_heads,
                                    int head_dim, size_t* bytes_out);

int pa_attention_int(void* out, const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                     const int32_t* query_start_loc, int num_seqs, int num_tokens, int max_query_len,
                     int max_seq_len, int num_heads, int num_kv_heads, int head_dim, int block_size,
                     int64_t num_blocks, float scale, int bits, void* workspace,
                     size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_attention_packed -- causal attention of prompts, or of chunks behind their contexts, over rows
 * that are at hand and need no pages: [docs] PagedAttention (the prompt's own attention), [flow] 3.2
 * and 3.5 (the flattened token batch), [intro] 2.1 (causal mask).
 *
 * Request s has the query rows [q_start_loc[s], q_start_loc[s + 1]) and the key and value rows
 * [k_start_loc[s], k_start_loc[s + 1]); with Q and K of them, query j sees keys 0 .. K - Q + j:
 *     out[q0 + j, h, :] = sum_i softmax_i(scale <q[q0 + j, h, :], k[k0 + i, g, :]>) v[k0 + i, g, :]
 * (h in KV head g's group); zeros where it sees none (j < Q - K).
 *
 * q, k, v       device, bf16, [num_q_rows, num_heads, head_dim] and [num_k_rows, num_kv_heads,
 *               head_dim]: token t's heads contiguous at q + t * q_stride elements (k_stride, v_stride
 *               alike), so that all three may be slices of one projection's output. Strides are multiples of
 *               16 bytes and at least the row; pointers 16-byte aligned
 * out           device, bf16 [num_q_rows, num_heads, head_dim], contiguous, apart from the inputs
 * q_start_loc, k_start_loc  device, int32 [num_seqs + 1], not decreasing. A request outside the rows, or
 *               of more than max_query_len queries, sets PA_DEVERR_SEQ_RANGE and its rows are left as they
 *               are; so are rows of no request
 * Numerators are rounded to bf16 for the second product, as pa_attention's are. A NaN or an infinity in
 * another request's rows changes nothing; one in a value row reaches the queries that see it and the
 * others of their tile: 128 / (num_heads / num_kv_heads) consecutive tokens, counted from the request's first.
 * Supported: head_dim 64 / 128, num_heads / num_kv_heads in {1, 2, 4, 8}, num_seqs <= 4096. One
 * launch on `stream`, no workspace.
 * --------------------------------------------------------------------------- */
int pa_attention_packed(void* out, const void* q, const void* k, const void* v, int64_t q_stride,
                        int64_t k_stride, int64_t v_stride, const int32_t* q_start_loc,
                        const int32_t* k_start_loc, int num_seqs, int num_q_rows, int num_k_rows,
                        int max_query_len, int num_heads, int num_kv_heads, int head_dim, float scale,
                        pa_dtype dtype, pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * pa_attention_fixed_scratch -- no counterpart in the pages: an addition for callers that
 * cannot allocate device memory, so cannot provide pa_attention's workspace. Examples: a
 * serving loop that reserved the GPU's free memory for its KV pool at start-up and must not
 * call cudaMalloc again (the call synchronises the device and fails once the pool owns the
 * memory); a plugin inside a host framework whose allocator it cannot reach; a binding from
 * a language with no device allocator.
 *
 * Same arguments and result as pa_attention, minus workspace / workspace_bytes, and with
 * every kernel on `stream` (no internal stream, so nothing is created). The split-K
 * scratch is instead a fixed 16 MiB array inside the library, which every GPU that loads
 * the library holds until the process exits. Allocates nothing (no cudaMalloc / cudaFree,
 * no allocating library call).
 *  - Limit: returns PA_ERR_WORKSPACE, enqueuing nothing, when the batch needs more scratch
 *    than 16 MiB (pa_attention_workspace_size gives the need; e.g. up to ~850 requests of
 *    32 query / 8 KV heads at head_dim 128 on a 152-SM GPU).
 *  - The first call on each device looks up the array's device address (once, with that
 *    device current); make that first call before any stream capture.
 *  - All calls on a device share the one array, which keeps the last call's contents; no
 *    part of it needs to start at zero. Calls whose work may overlap on the GPU (different
 *    streams without ordering between them) race on it and give wrong results: order them.
 * --------------------------------------------------------------------------- */
int pa_attention_fixed_scratch(void* out, const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, int max_blocks_per_seq,
                               const int32_t* seq_lens, const int32_t* query_start_loc,
                               int num_seqs, int num_tokens, int max_query_len, int max_seq_len,
                               int num_heads, int num_kv_heads, int head_dim, int block_size,
                               int64_t num_blocks, float scale, pa_dtype dtype,
                               pa_stream_t stream);

/* ------------------------------------------------------------------------------
 * Host block manager -- [docs] PagedAttention algorithm flow and Copy-on-Write
 * (reference counting); [read] 5.1.1 and 5.2.1; [flow] 3.3 (pool of blocks, slots).
 *
 * Free blocks are handed out first-in first-out, starting from `free_order` (a
 * permutation of [0, num_blocks)); a released block rejoins the tail (the free list is
 * doubly linked so that prefix caching, below, can take a released block back out). Appending a
 * token takes a new block only when the sequence's last block is full (or it has none),
 * so a sequence of n tokens holds ceil(n / block_size) blocks. Writing into a last
 * block whose reference count is > 1 first moves the writer to a fresh block and
 * records a (src, dst) copy pair; the old block's count drops by 1. An append that
 * cannot be satisfied changes nothing. Not thread-safe: one manager per thread.
 * All arrays are host memory.
 * --------------------------------------------------------------------------- */
typedef struct pa_bm pa_bm;

/* NULL on invalid arguments (free_order not a permutation, sizes < 1) or no memory. */
pa_bm* pa_bm_create(int64_t num_blocks, int block_size, const int32_t* free_order);
void pa_bm_destroy(pa_bm* bm);

int pa_bm_add_seq(pa_bm* bm, int64_t seq);               /* PA_ERR_NOT_FOUND if id in use */
/* Appends n >= 0 tokens; writes their n slots to slots_out (may be NULL when n == 0).
 * PA_ERR_NO_BLOCKS: the free queue is too short now; PA_ERR_TOO_LARGE: the sequence
 * would need more blocks than the pool has. */
int pa_bm_append(pa_bm* bm, int64_t seq, int64_t n, int64_t* slots_out);
/* Batched append: for i in [0, n), appends counts[i] >= 0 tokens to seqs[i], in order, writing
 * all slots concatenated to slots_out (capacity >= sum of counts). Stops at the first append
 * that fails and returns its status; *done_out (if not NULL) gets the number of entries fully
 * applied, so those appends stay and the rest are not attempted. */
int pa_bm_append_batch(pa_bm* bm, const int64_t* seqs, const int64_t* counts, int64_t n,
                       int64_t* slots_out, int64_t* done_out);
int pa_bm_fork(pa_bm* bm, int64_t parent, int64_t child); /* child shares parent's blocks */
int pa_bm_free_seq(pa_bm* bm, int64_t seq);               /* counts - 1, release at 0 */
int64_t pa_bm_seq_len(const pa_bm* bm, int64_t seq);      /* -1 if unknown */
int64_t pa_bm_num_seq_blocks(const pa_bm* bm, int64_t seq);/* -1 if unknown */
int pa_bm_ref_count(const pa_bm* bm, int64_t block);      /* -1 if out of range */
int64_t pa_bm_num_free(const pa_bm* bm);
/* Copies the free queue, head first, into out (capacity >= pa_bm_num_free). */
int pa_bm_free_queue(const pa_bm* bm, int32_t* out, int64_t capacity);
/* Copies seq's block table (logical order) into out (capacity >= its block count). */
int pa_bm_block_table(const pa_bm* bm, int64_t seq, int32_t* out, int64_t capacity);
/* Fills a batch's metadata: row i of table_out [n, width] gets seqs[i]'s block table
 * (unused entries 0) and seq_lens_out[i] its length. PA_ERR_INVALID_ARG if a table is
 * wider than `width`. */
int pa_bm_batch_tables(const pa_bm* bm, const int64_t* seqs, int64_t n, int32_t* table_out,
                       int64_t width, int32_t* seq_lens_out);
int64_t pa_bm_num_pending_copies(const pa_bm* bm);
/* Moves up to `capacity` pending (src, dst) pairs, oldest first, into pairs_out
 * [capacity, 2]; returns how many were moved (or -1 on a bad argument). */
int64_t pa_bm_take_copies(pa_bm* bm, int64_t* pairs_out, int64_t capacity);

/* ------------------------------------------------------------------------------
 * Prefix caching -- [docs] Copy-on-Write › shared-prefix detection (hash a prompt's
 * prefix; if its KV is cached, reuse it and raise the blocks' reference counts) and
 * Prefix Caching › mechanism (look up on arrival; a hit reuses the KV and skips that
 * prefill, a miss computes and caches it); [flow] 3.3 (blocks on a doubly linked list,
 * evicted least recently used first).
 *
 * Once enabled, a full block is keyed by its whole token prefix (all token ids of its
 * sequence up to its last slot; a 128-bit hash chain encodes it). A block is registered
 * when its last slot is written, unless its key is registered already (the first block
 * stays registered). A released block keeps its registration at the tail of the free
 * list; the free list hands blocks out from its head, and a registered block handed out
 * loses its registration (eviction, least recently released first). Cached blocks are
 * full, so nothing ever writes into them while they are shared.
 * --------------------------------------------------------------------------- */
/* Turns prefix caching on; only on a fresh manager (no sequence yet). From then on appends
 * need token ids: pa_bm_append / pa_bm_append_batch return PA_ERR_INVALID_ARG. */
int pa_bm_enable_prefix_caching(pa_bm* bm);
/* Starts sequence `seq` from the longest cached prefix of prompt[0, n): whole blocks, walked
 * from the start until the first miss, covering at most max_hit tokens (pass n - 1 so the
 * last prompt token is always computed). The reused blocks' counts go up (a released one
 * leaves the free list). *hit_out = tokens reused (a multiple of block_size); the caller
 * appends prompt[*hit_out, n) next and computes only those rows. */
int pa_bm_add_seq_cached(pa_bm* bm, int64_t seq, const int32_t* prompt, int64_t n, int64_t max_hit,
                         int64_t* hit_out);
/* pa_bm_append with the appended tokens' ids (token_ids[n]; ignored without caching). */
int pa_bm_append_tokens(pa_bm* bm, int64_t seq, const int32_t* token_ids, int64_t n, int64_t* slots_out);
/* pa_bm_append_batch with token ids, concatenated like the slots. */
int pa_bm_append_tokens_batch(pa_bm* bm, const int64_t* seqs, const int64_t* counts, int64_t n,
                              const int32_t* token_ids, int64_t* slots_out, int64_t* done_out);
/* Registered blocks now, blocks reused by lookups so far, registrations evicted so far. */
int pa_bm_prefix_stats(const pa_bm* bm, int64_t* cached_blocks, int64_t* hit_blocks, int64_t* evictions);

/* Groups for pa_attention_grouped over the batch seqs[0, n) (in batch order): runs of
 * consecutive sequences whose block tables start with the same block id, at most
 * max_members each, become groups; shared_len = the number of leading table entries all
 * members have in common x block_size, capped by the shortest member. Writes
 * seq_group_out[n] (-1 outside groups), group_range_out[2 * groups] and
 * shared_len_out[groups] (capacity >= n / 2 groups is always enough) and *num_groups_out. */
int pa_bm_batch_groups(const pa_bm* bm, const int64_t* seqs, int64_t n, int max_members, int32_t* seq_group_out,
                       int32_t* group_range_out, int32_t* shared_len_out, int64_t capacity,
                       int64_t* num_groups_out);

/* ------------------------------------------------------------------------------
 * Swapping -- [read] 6.2.1 SequenceGroup (preempted groups are swapped out to the CPU and
 * swapped back in later); [intro] 4, scheduling flow, swap phase (swapped queue in CPU
 * memory).
 *
 * A CPU pool of num_cpu_blocks blocks with its own FIFO free queue (initial order
 * cpu_free_order) and reference counts. pa_bm_swap_out moves a group of sequences to the
 * CPU: each distinct block of their tables (first met walking seqs in order, each table
 * from its first block) gets one CPU block whose count is the number of group members
 * holding it; the GPU block's count drops by that number and it is released at 0 (a block
 * still held outside the group stays). The (gpu, cpu) pairs to copy go to pairs_out
 * [capacity, 2] and their number to *num_pairs_out; run pa_swap_blocks with them before
 * the released GPU blocks are written again. pa_bm_swap_in is the reverse (new GPU
 * blocks from the free list, (cpu, gpu) pairs; copy them before reading the sequences).
 * Either returns PA_ERR_NO_BLOCKS (changing nothing) when the other pool is short,
 * PA_ERR_INVALID_ARG when capacity is below the number of pairs, a sequence repeats or is
 * already on the other side. A swapped sequence takes no append or fork and cannot be in
 * pa_bm_batch_tables; pa_bm_free_seq releases its CPU blocks.
 * --------------------------------------------------------------------------- */
int pa_bm_enable_swap(pa_bm* bm, int64_t num_cpu_blocks, const int32_t* cpu_free_order);
int pa_bm_swap_out(pa_bm* bm, const int64_t* seqs, int64_t n, int64_t* pairs_out, int64_t capacity,
                   int64_t* num_pairs_out);
int pa_bm_swap_in(pa_bm* bm, const int64_t* seqs, int64_t n, int64_t* pairs_out, int64_t capacity,
                  int64_t* num_pairs_out);
int pa_bm_is_swapped(const pa_bm* bm, int64_t seq);        /* 1, 0, or -1 if unknown */
int64_t pa_bm_num_free_cpu(const pa_bm* bm);               /* -1 without swapping */
int pa_bm_cpu_ref_count(const pa_bm* bm, int64_t block);  /* -1 if out of range */

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
