/*
 * pagedattn.h — C ABI of libpagedattn.so, paged decode attention for NVIDIA B200 (sm_100a).
 *
 * Scope: the decode-step hot path of PagedAttention. The KV cache is cut into fixed-size
 * blocks (8, 16 or 32 tokens; 16 by default) scattered through a physical block pool; a per-sequence block table maps
 * logical blocks to physical ones; sequences with a common prefix share physical blocks,
 * counted by ref_count, and a shared block is copied before it is written (copy-on-write).
 * Sources (page title, section):
 *   [KVPaged] "KV cache and paged attention" (youngju.dev)
 *   [Ch4PA]   "Why PagedAttention cuts GPU memory waste by up to 95%" (iq-universe.github.io,
 *             ch4-paged-attention)
 *   [OpsVLLM] "How does vLLM PagedAttention manage the KV cache" (opsoai.com)
 *   [KVFail]  "Transformer inference KV-cache memory-management failure modes"
 *             (knowledge.openakashic.com)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers named *_cache, q, out, k, v, block_tables, context_lens, query_start,
 *   slot_mapping, pairs, *_scales, *_zeros, lse_out and workspace are DEVICE pointers; the
 *   caller owns them. The library allocates no device memory (paged_attn_decode_noalloc's
 *   fixed array is compiled into the library, below).
 * - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Device
 *   work is enqueued asynchronously on it; a PA_OK return means "enqueued".
 * - Every call validates its host-side arguments first and returns an error without
 *   enqueuing anything when they are wrong. Faults of asynchronous work show up at the next
 *   synchronisation, as with any CUDA launch.
 * - Data that lives on the device cannot be validated by the host. Kernels bounds-check
 *   every block id, slot and copy pair they read; an out-of-range value is skipped (the
 *   access is not made) and recorded in a device error word, see pa_device_error().
 * - Cache layout: cache[num_blocks][num_kv_heads][block_size][head_dim], row-major, so each
 *   (physical block, kv head) tile is contiguous (the pages give no layout; this is the
 *   library's choice). fp8 caches carry float32 scales[num_blocks][num_kv_heads], one per
 *   (block, kv head), separately for K and V: stored value = E4M3(x / scale). int8 caches
 *   ([KVPaged] "KV quantization: FP8 and INT8": one byte per element with a scale and a
 *   zero point) carry the same scales plus int32 zero points[num_blocks][num_kv_heads]:
 *   stored code = clamp(round_half_even(x / scale) + zero, -128, 127), value =
 *   (code - zero) * scale. Zero points must lie in [-128, 127], the byte's own range
 *   (an affine int8 code needs no other); there code - zero is exact in every kernel. A
 *   block whose K or V zero point lies outside is treated like a bad block id: attention
 *   skips it and the cache write skips its rows, and PA_DEVERR_ZERO is recorded.
 * - q and out: [num_seqs][num_q_heads][head_dim] row-major. Query head h reads kv head
 *   h / (num_q_heads / num_kv_heads) ([KVPaged] "GQA and MQA": query heads are grouped and
 *   each group shares one KV head).
 * - block_tables: int32 [num_seqs][max_blocks_per_seq]; entry b of row s is the physical
 *   block holding logical tokens [B*b, B*b+B) of sequence s (B = block_size); entries at or beyond
 *   ceil(context_lens[s] / block_size) are never read ([Ch4PA] "PagedAttention algorithm":
 *   the block table maps logical block ids to physical blocks that need not be contiguous).
 * - context_lens[s] counts every cached token of sequence s, including the token being
 *   decoded (whose K/V must have been written by reshape_and_cache first).
 *
 * Supported today: block_size 8, 16 or 32 ([KVPaged] "the block-size knob" and [Ch4PA]
 * "Theorem 1, fragmentation bound": smaller blocks waste less of the last block, larger
 * ones need shorter tables; 16 is the usual default); head_dim 64, 128 or 256; num_q_heads a multiple of
 * num_kv_heads with a group of at most 16; (q, kv, out) dtypes (f32, f32, f32),
 * (bf16, bf16, bf16), (bf16, fp8_e4m3, bf16) and (bf16, int8, bf16). Anything else returns
 * PA_ERR_UNSUPPORTED.
 */
#ifndef PAGEDATTN_H_
#define PAGEDATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2, PA_INT8 = 3 } pa_dtype;

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID = -1,      /* bad argument: null pointer, size out of range, bad id      */
  PA_ERR_UNSUPPORTED = -2,  /* valid but not implemented (dtype combination, head_dim...) */
  PA_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed                       */
  PA_ERR_NO_BLOCKS = -4,    /* allocator: not enough free blocks; nothing was changed     */
  PA_ERR_WORKSPACE = -5,    /* workspace missing or smaller than paged_attn_workspace_size */
  PA_ERR_DEVICE = -6        /* a kernel recorded a bad block id / slot / pair, see below  */
} pa_status;

/* Bits of the device error word (pa_device_error). */
#define PA_DEVERR_BLOCK_ID 0x1   /* block table entry outside [0, num_blocks)          */
#define PA_DEVERR_SLOT 0x2       /* slot_mapping entry outside [-inf, num_blocks*bs)    */
#define PA_DEVERR_PAIR 0x4       /* copy_blocks pair outside [0, num_blocks)            */
#define PA_DEVERR_CONTEXT 0x8    /* context_lens entry < 0 or > max_context_len         */
#define PA_DEVERR_TIMEOUT 0x10   /* a bounded wait on an asynchronous copy gave up      */
#define PA_DEVERR_QUERY 0x20     /* prefill query_start not ascending, past num_tokens, */
                                 /* or more new tokens than context (or max_query_len)  */
#define PA_DEVERR_ZERO 0x40      /* int8 zero point outside [-128, 127]                 */
#define PA_DEVERR_TREE 0x80      /* draft tree: parent not before its child, more than  */
                                 /* the mask's (or 256) tokens, bad accepted path       */
#define PA_DEVERR_BLOCKS 0x100   /* device free queue shorter than a step's new blocks  */
#define PA_DEVERR_QUEUE 0x200    /* device free queue: head or count out of range, or   */
                                 /* more blocks returned than the ring holds            */

/*
 * partition_size value that lets the library choose the split for a decode call: one
 * pass (0) when max_context_len <= 512; else 512 tokens when num_seqs * num_kv_heads >=
 * 1024, else 1024. The choice depends only on the descriptor and max_context_len, so
 * results stay independent of where blocks sit; paged_attn_partition_size() reports it.
 */
#define PA_PARTITION_AUTO (-1)

/* Shape and dtypes of one paged decode-attention call. */
typedef struct {
  int num_seqs;            /* S >= 0                                                   */
  int num_q_heads;         /* Hq                                                       */
  int num_kv_heads;        /* Hkv; Hq % Hkv == 0                                       */
  int head_dim;            /* d                                                        */
  int block_size;          /* tokens per block: 8, 16 or 32                            */
  int max_blocks_per_seq;  /* row stride of block_tables                               */
  int num_blocks;          /* physical blocks in the pool (bounds check)               */
  int partition_size;      /* split-KV partition in tokens, a multiple of block_size   */
                           /* and of 16;                                               */
                           /* 0 = one pass over the whole context per (seq, kv head);  */
                           /* PA_PARTITION_AUTO = the library's choice (below)         */
  pa_dtype q_dtype, kv_dtype, out_dtype;
} pa_decode_desc;

/*
 * Bytes of device workspace paged_attn_decode needs for this shape when no context is
 * longer than max_context_len (0 when partition_size == 0). Returns 0 for an invalid
 * descriptor as well; paged_attn_decode then reports the error.
 */
size_t paged_attn_workspace_size(const pa_decode_desc* desc, int max_context_len);

/*
 * The partition (tokens; 0 = one pass) a paged_attn_decode call with this descriptor uses:
 * desc->partition_size itself, or the library's choice for PA_PARTITION_AUTO. -1 for an
 * invalid descriptor.
 */
int paged_attn_partition_size(const pa_decode_desc* desc, int max_context_len);

/*
 * Number of kernel launches one paged_attn_decode call with this descriptor makes under
 * the current pa_set_decode_impl choice (0 for an invalid, unsupported or empty call):
 * the plan kernel of the persistent tensor-core kernels, the attention kernel, and the
 * log-sum-exp reduce when the split path's partitions are not merged in place. For
 * callers that count launches (profiling, launch budgets).
 */
int paged_attn_decode_launches(const pa_decode_desc* desc, int max_context_len);

/*
 * Decode attention over the paged cache ([KVPaged] "Core principle: what is the KV cache":
 * attention(Q,K,V) = softmax(Q K^T / sqrt(d_k)) V, one new query per sequence; [Ch4PA]
 * "PagedAttention algorithm": the kernel looks every logical block up in the block table
 * and gathers the non-contiguous K and V blocks). For every sequence s and query head h,
 * with g = h / (Hq/Hkv) and the cached tokens t < context_lens[s]:
 *     z_t = scale * q[s][h] . K_t,   out[s][h] = sum_t softmax(z)_t V_t,
 *     lse_out[s][h] = log sum_t exp(z_t)                    (natural log, float32)
 * fp8 caches are dequantised as E4M3 value * scales[block][g], int8 caches as
 * (code - zeros[block][g]) * scales[block][g]. Accumulation is float32.
 * With partition_size > 0 the context is cut into partitions of that many logical tokens,
 * each reduced to (max, sum, unnormalised output) in `workspace`, then combined by a
 * log-sum-exp reduction; the result does not depend on where blocks sit physically.
 *   q, out         [S][Hq][d] in desc->q_dtype / desc->out_dtype
 *   k_cache/v_cache pool in desc->kv_dtype (layout above)
 *   block_tables   int32 [S][max_blocks_per_seq];  context_lens int32 [S]
 *   max_context_len  host int >= every context_lens entry (sizes the grid)
 *   k_scales/v_scales float32 [num_blocks][Hkv], required for fp8 and int8, else ignored
 *   k_zeros/v_zeros  int32 [num_blocks][Hkv], required for int8, ignored otherwise
 *   lse_out        float32 [S][Hq] or NULL
 *   workspace      device bytes, >= paged_attn_workspace_size(desc, max_context_len),
 *                  16-byte aligned; may be NULL when that size is 0
 * A sequence with context length 0 gets out = 0 and lse = -inf.
 */
pa_status paged_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens,
                            float scale, void* out, const pa_decode_desc* desc,
                            int max_context_len, const float* k_scales, const float* v_scales,
                            const int32_t* k_zeros, const int32_t* v_zeros, float* lse_out,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Prefill attention over the paged cache: the new tokens of a step attend causally to
 * their sequence's cached tokens ([KVPaged] "Core principle: what is the KV cache": the
 * prompt's K/V is computed once and cached, each token attending to itself and all earlier
 * tokens; "Prefix sharing and copy-on-write": a cached prefix's K/V is computed once, so
 * a step may bring only the tokens after it, as may a prompt cut into chunks). Sequence s
 * brings n_s = query_start[s+1] - query_start[s] new tokens, rows query_start[s] .. of q,
 * whose K/V were written by reshape_and_cache first as the last n_s of its
 * context_lens[s] positions. Row i of sequence s sits at position p = context_lens[s] -
 * n_s + i; for query head h (kv head g = h / (Hq/Hkv)):
 *     z_t = scale * q[row][h] . K_t (t <= p),  out[row][h] = sum_t softmax(z)_t V_t,
 *     lse_out[row][h] = log sum_t exp(z_t)              (natural log, float32)
 * with fp8 / int8 dequantisation as in paged_attn_decode. Accumulation is float32.
 *   q, out        [num_tokens][Hq][d] in desc->q_dtype / desc->out_dtype
 *   query_start   int32 [num_seqs + 1], ascending, query_start[0] = 0,
 *                 query_start[num_seqs] = num_tokens
 *   max_query_len host int >= every n_s (sizes the grid); max_context_len >= every
 *                 context_lens entry and >= max_query_len
 *   block_tables, context_lens, k/v scales and zeros, lse_out: as in paged_attn_decode
 *   desc          as in paged_attn_decode with partition_size 0
 * bf16 q / out with a bf16, fp8 or int8 cache, head_dim 128 and a group of 1, 2, 4, 8 or
 * 16 run on the tensor cores (tcgen05, accumulators in tensor memory; fp8 / int8 codes are
 * converted exactly to bf16 in shared memory and their scales applied to the scores and
 * to P); every other supported shape, or pa_set_decode_impl(1), runs one CUDA-core pass
 * per new token. No workspace.
 * A sequence whose query range is inconsistent (descending, past num_tokens, more new
 * tokens than context or than max_query_len) is skipped and PA_DEVERR_QUERY recorded.
 */
pa_status paged_attn_prefill(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* query_start, int num_tokens, int max_query_len,
                             float scale, void* out, const pa_decode_desc* desc,
                             int max_context_len, const float* k_scales, const float* v_scales,
                             const int32_t* k_zeros, const int32_t* v_zeros, float* lse_out,
                             void* stream);

/*
 * Largest workspace (bytes) that paged_attn_decode_noalloc can serve from its fixed device
 * array: 32 MiB.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * paged_attn_decode for callers that cannot allocate device memory. Some callers may not
 * call cudaMalloc at all: a plugin inside a host runtime that owns every device allocation
 * through its own allocator, a caller with no workspace argument to forward, a latency-
 * bound loop that must not risk cudaMalloc's implicit device synchronisation. This entry
 * point takes the same arguments as paged_attn_decode minus the workspace and computes the
 * same result, bit for bit; the split-KV scratch comes from one fixed array compiled into
 * this library (PA_NOALLOC_SCRATCH_BYTES per GPU, held by every GPU that loads the library
 * until the process exits). The pages have no counterpart of this call; it exists only for
 * such callers.
 * - Calls that need more scratch than PA_NOALLOC_SCRATCH_BYTES
 *   (paged_attn_workspace_size(desc, max_context_len) larger than it) return
 *   PA_ERR_WORKSPACE and enqueue nothing.
 * - The first call on a device, whatever its shape, looks the array's device address up
 *   (once per device, with that device current); make that first call before any stream
 *   capture.
 * - It calls no cudaMalloc, cudaFree or other allocating routine.
 * - Every call on a device shares the one array, which keeps the last call's contents. The
 *   kernels re-initialise what they read (work counter, partials) on every call, so stale
 *   contents never matter; but calls that overlap on the GPU (different streams, or
 *   different host threads) race on the array: serialise them.
 */
pa_status paged_attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    float scale, void* out, const pa_decode_desc* desc,
                                    int max_context_len, const float* k_scales,
                                    const float* v_scales, const int32_t* k_zeros,
                                    const int32_t* v_zeros, float* lse_out, void* stream);

/*
 * Slot-mapped write of new tokens' K and V into the pool ([KVPaged] "PagedAttention: OS
 * virtual-memory style management": one block is allocated as tokens accumulate and the
 * block table maps logical positions to physical blocks). For token t with
 * slot = slot_mapping[t] >= 0, block = slot / block_size, offset = slot % block_size:
 *     k_cache[block][h][offset][:] = convert(k[t][h][:])   for every kv head h (same for v)
 * convert: f32->f32 and bf16->bf16 copy bits; f32->bf16 rounds to nearest even; f32 or
 * bf16 -> fp8 stores E4M3(x / scale[block][h]) with an IEEE float32 division, round to
 * nearest even, saturating to +-448; f32 or bf16 -> int8 stores
 * clamp(round_half_even(x / scale[block][h]) + zero[block][h], -128, 127), same division.
 * A negative slot is a padding token and is skipped.
 *   k, v             device [num_tokens][Hkv][head_dim] rows, token stride k_stride /
 *                    v_stride elements (>= Hkv*head_dim), in in_dtype
 *   slot_mapping     int64 [num_tokens]
 *   k_scales/v_scales float32 [num_blocks][Hkv], fp8 and int8 caches (read, not written)
 *   k_zeros/v_zeros  int32 [num_blocks][Hkv], int8 caches only (read, not written)
 * Tokens must map to distinct slots (two writes to one slot race).
 */
pa_status reshape_and_cache(const void* k, const void* v, void* k_cache, void* v_cache,
                            const int64_t* slot_mapping, int num_tokens, int64_t k_stride,
                            int64_t v_stride, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, pa_dtype in_dtype, pa_dtype cache_dtype,
                            const float* k_scales, const float* v_scales,
                            const int32_t* k_zeros, const int32_t* v_zeros, void* stream);

/*
 * Copy-on-write block copy ([KVPaged] "Prefix sharing and copy-on-write": a shared block is
 * copied before one sharer modifies it; [Ch4PA] "Prefix Caching": copies happen only on
 * write). For each pair i, (src, dst) = (pairs[2i], pairs[2i+1]) (device int32 [n][2]):
 * the K and V tiles of every kv head of block src are copied to block dst, and for fp8
 * and int8 caches the scales too (k_scales/v_scales may be NULL otherwise), for int8 also
 * the zero points (k_zeros/v_zeros may be NULL otherwise). No dst may appear twice
 * or also be a src: such copies race. Enqueue it before the reshape_and_cache that writes
 * into the destination blocks.
 */
pa_status copy_blocks(void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                      int32_t* k_zeros, int32_t* v_zeros, const int32_t* pairs, int num_pairs,
                      int num_kv_heads, int head_dim, int block_size, int num_blocks,
                      pa_dtype cache_dtype, void* stream);

/* ------------------------------------------------------------------------------------- */
/* A drafted (speculative) step on the GPU. Several tokens per sequence are drafted ahead  */
/* as a tree, checked by the model in one step and the longest agreeing path is kept. Each */
/* step extends the block tables and maps slots (paged_build_step), rotates q and k and    */
/* writes the cache (rotary_and_cache), attends from the tree (paged_attn_tree), picks the */
/* accepted path (tree_verify) and moves its K/V behind the context (compact_accepted).    */
/* Nothing of it needs the host, so a step can be captured in a CUDA graph.                */
/*                                                                                        */
/* Trees: sequence s drafts n_s tokens, rows query_start[s] .. query_start[s+1]-1 of the    */
/* step. parents[row] is the index within the sequence (0 .. n_s-1) of the row's parent,  */
/* smaller than the row's own index, or -1 for a row right behind the context. Row 0 is   */
/* the sequence's newest known token, whose K/V is not cached yet; rows behind it are     */
/* drafts. Row i sees the cached context, its ancestors and itself: bit j % 32 of word     */
/* j / 32 of its mask is set when it sees row j. At most 256 rows per sequence.           */
/* ------------------------------------------------------------------------------------- */
/*
 * A step's block tables, slot map and positions from request lengths ([KVPaged]
 * "PagedAttention: OS virtual-memory style management": one block is taken as tokens
 * accumulate; [KVFail] Key Points: blocks come from a free queue and a step fails when too
 * few are free). Sequence s holds blocks_held[s] blocks (the first entries of its row of
 * block_tables) and context_lens[s] cached tokens, and brings new_lens[s] tokens. In
 * sequence order, each takes max(0, ceil((context + new) / block_size) - held) blocks from
 * the front of the free queue: the blocks pa_alloc_append_batch would take in the same
 * state when no block is shared. A partially filled last block must not be shared
 * (pa_alloc_append copies such a block; this call does not).
 *   context_lens, new_lens, blocks_held   device int32 [num_seqs]
 *   parents          device int32 [max_tokens] or NULL (every row the child of the row
 *                    before it); rows behind the last sequence are not read
 *   block_tables     device int32 [num_seqs][max_blocks_per_seq]; the new entries are written
 *   free_blocks      device int32 [free_capacity], a ring of free block ids
 *   queue_state      device int32 [2]: index of the ring's front, number of free blocks
 *   total_lens       out, int32 [num_seqs]: context + new
 *   query_start      out, int32 [num_seqs + 1]: each sequence's first row, then their number
 *   blocks_held_out, queue_state_out      out, as the inputs, after this step
 *   slot_mapping     out, int64 [max_tokens]: slot of row i of sequence s, at position
 *                    context + i; -1 for rows behind the last sequence
 *   positions        out, int32 [max_tokens] or NULL: context + number of the row's
 *                    ancestors (context + i without parents); 0 behind the last sequence
 *   tree_mask        out, uint32 [max_tokens][mask_words] or NULL; 0 behind the last sequence
 *   mask_words       1 to 8 when tree_mask is given (new_lens at most 32 * mask_words)
 *   status           out, int32 [1] or NULL: 0, or the PA_DEVERR_* bits that made it fail
 * All or nothing: a negative length, a table too short or held blocks fewer than the
 * context needs (PA_DEVERR_CONTEXT), more tokens than max_tokens (PA_DEVERR_QUERY), more
 * than the mask holds (PA_DEVERR_TREE), a bad queue state (PA_DEVERR_QUEUE) or too few free
 * blocks (PA_DEVERR_BLOCKS) leave tables, held blocks and queue as they were, and give a
 * step of no tokens: query_start and masks 0, every slot -1, total_lens = context_lens. A bad
 * parent is recorded (PA_DEVERR_TREE) and its row treated as one right behind the context;
 * a row whose block id is outside [0, num_blocks) gets slot -1 (PA_DEVERR_BLOCK_ID).
 * Every output but block_tables is written in full; none may overlap an input. The same
 * call on the same inputs gives the same outputs. That holds for num_seqs = 0 too (an idle
 * step: no rows, every slot -1, the queue passed on); the buffers of one entry per sequence
 * may then be NULL. Only a call of no sequences that has new_lens and no context_lens is
 * taken for no batch at all: PA_OK, nothing is written.
 */
pa_status paged_build_step(const int32_t* context_lens, const int32_t* new_lens,
                           const int32_t* blocks_held, const int32_t* parents,
                           int32_t* block_tables, const int32_t* free_blocks,
                           const int32_t* queue_state, int num_seqs, int max_blocks_per_seq,
                           int block_size, int num_blocks, int free_capacity, int max_tokens,
                           int mask_words, int32_t* total_lens, int32_t* query_start,
                           int32_t* blocks_held_out, int32_t* queue_state_out,
                           int64_t* slot_mapping, int32_t* positions, uint32_t* tree_mask,
                           int32_t* status, void* stream);

/*
 * Returns blocks to the back of the device free queue: sequence s keeps its first
 * min(held, ceil(keep_lens[s] / block_size)) blocks, the others go to the queue in sequence
 * order and, within one, in table order (the order of pa_alloc_free_seq). keep_lens[s] = 0
 * ends a sequence; its context length returns blocks of drafts that were not accepted.
 * Blocks of a sequence that shares them must not be returned here. Table entries stay as
 * they are (blocks_held_out says how many count). Buffers as in paged_build_step;
 * free_blocks is written. All or nothing: a negative length, held blocks outside [0,
 * max_blocks_per_seq] (PA_DEVERR_CONTEXT) or a queue that would not hold them
 * (PA_DEVERR_QUEUE) change nothing but the outputs, which are as the inputs. num_seqs = 0
 * passes the queue on, with buffers as in paged_build_step (no batch at all: blocks_held
 * and no keep_lens).
 */
pa_status paged_release_blocks(const int32_t* keep_lens, const int32_t* blocks_held,
                               const int32_t* block_tables, int32_t* free_blocks,
                               const int32_t* queue_state, int num_seqs,
                               int max_blocks_per_seq, int block_size, int free_capacity,
                               int32_t* blocks_held_out, int32_t* queue_state_out,
                               int32_t* status, void* stream);

/* Shape, strides and types of one rotary_and_cache call. */
typedef struct {
  int num_tokens, num_q_heads, num_kv_heads;
  int head_dim;             /* 64, 128 or 256                                             */
  int rotary_dim;           /* leading channels that are rotated: a multiple of 16, at     */
                            /* most head_dim                                              */
  int num_axes;             /* 1 to 4 position axes                                       */
  int sections[4];          /* frequencies of each axis, in order; sum = rotary_dim / 2    */
  int adjacent_pairs;       /* 0: channel i turns with i + rotary_dim / 2; 1: 2i with 2i+1 */
  int block_size, num_blocks;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  /* elements from token to token     */
  pa_dtype in_dtype;        /* q, k, v and q_out: PA_F32 or PA_BF16                        */
  pa_dtype cache_dtype;
} pa_rotary_desc;

/*
 * Rotary positions on q and k, fused with the slot-mapped cache write of k and v. Frequency
 * i of token t turns the pair (x, y) of its two channels by the angle positions[axis][t] *
 * inv_freq[i], axis being the one whose section holds i (time, height and width of image and
 * video tokens; one axis for text):  x' = x cos - y sin, y' = y cos + x sin.
 * The angle is formed and reduced in float64, so far positions lose nothing; products are
 * float32. q_out gets the turned q rounded once to in_dtype; the cache gets the turned k and
 * v, converted as reshape_and_cache does but from float32, with no rounding in between.
 *   q, k, v, q_out   rows [heads][head_dim], token strides in the descriptor; q_out may be
 *                    q itself
 *   positions        int32 [num_axes][num_tokens]
 *   slot_mapping     int64 [num_tokens]; a negative slot is a padding token: nothing of it
 *                    is read or written (its q_out row stays as it was)
 *   inv_freq         float32 [rotary_dim / 2]
 *   k_scales ..      as in reshape_and_cache
 * Types as in reshape_and_cache. Tokens must map to distinct slots.
 */
pa_status rotary_and_cache(const void* q, const void* k, const void* v, void* q_out,
                           void* k_cache, void* v_cache, const int32_t* positions,
                           const int64_t* slot_mapping, const float* inv_freq,
                           const pa_rotary_desc* desc, const float* k_scales,
                           const float* v_scales, const int32_t* k_zeros,
                           const int32_t* v_zeros, void* stream);

/* Bytes of device workspace paged_attn_tree needs (0 for an invalid or empty call). */
size_t paged_attn_tree_workspace_size(const pa_decode_desc* desc, int num_tokens,
                                      int max_query_len, int max_context_len);

/*
 * Attention of a step's drafted tokens over the paged cache. As paged_attn_prefill, except
 * that row i of sequence s, whose n_s rows are the last n_s of its context_lens[s]
 * positions, sees every position before context_lens[s] - n_s and, of the rows
 * themselves, those whose bit is set in its mask (which may be none: a row that sees
 * nothing at all gets out = 0 and lse = -inf). The masks are taken as they are; they need
 * not be a tree's.
 *   tree_mask        uint32 [num_tokens][mask_words], mask_words 1 to 8
 *   max_query_len    host int >= every n_s, at most 32 * mask_words
 *   desc             as in paged_attn_decode, partition_size 0 or PA_PARTITION_AUTO (the
 *                    library splits long contexts and joins the parts)
 *   workspace        device bytes, >= paged_attn_tree_workspace_size(...), 16-byte aligned;
 *                    calls that overlap on the GPU need one each
 * Other arguments and errors as in paged_attn_prefill. bf16 q / out with head_dim 128 and a
 * group of 1, 2, 4, 8 or 16 run on the tensor cores; other shapes, or
 * pa_set_decode_impl(1), on the CUDA cores. Rows behind query_start[num_seqs] are neither
 * read nor written. Results depend on lengths and values, not on where blocks sit.
 * Precision: sums, softmax statistics and the joining of parts are float32 everywhere. The
 * tensor cores multiply V by weights rounded to bf16 for a bf16 cache (2^-8 relative), to f16
 * for one-byte caches (2^-11); the CUDA cores round nothing but the output.
 * max_context_len also sets how contexts are cut over the GPU: a limit far above the lengths
 * in the batch gives the same results, later.
 */
pa_status paged_attn_tree(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens,
                          const int32_t* query_start, const uint32_t* tree_mask,
                          int mask_words, int num_tokens, int max_query_len, float scale,
                          void* out, const pa_decode_desc* desc, int max_context_len,
                          const float* k_scales, const float* v_scales, const int32_t* k_zeros,
                          const int32_t* v_zeros, float* lse_out, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * The accepted path of each sequence's draft tree under greedy choice: from row 0, whose
 * token is known, go to the child (lowest index first) whose drafted token is the one the
 * model chose after its parent, until none agrees or max_accept rows are taken.
 *   parents, query_start       as above; context_lens int32 [num_seqs], the rows included
 *   draft_tokens     int64 [num_tokens]: token of each row
 *   target_tokens    int64 [num_tokens]: the model's choice after each row
 *   accepted         out, int32 [num_seqs][max_accept]: rows of the path, ascending, then -1
 *   num_accepted     out, int32 [num_seqs]
 *   next_tokens      out, int64 [num_seqs]: the model's choice after the last accepted row
 *   kept_lens        out, int32 [num_seqs]: context without drafts + num_accepted
 * A sequence without rows gets 0 accepted, next token -1 and kept_lens = context_lens; so does one whose
 * range is inconsistent (PA_DEVERR_QUERY) or longer than 256 rows (PA_DEVERR_TREE).
 */
pa_status tree_verify(const int32_t* parents, const int64_t* draft_tokens,
                      const int64_t* target_tokens, const int32_t* query_start,
                      const int32_t* context_lens, int num_seqs, int num_tokens,
                      int max_accept, int32_t* accepted, int32_t* num_accepted,
                      int64_t* next_tokens, int32_t* kept_lens, void* stream);

/*
 * Moves the K/V of accepted rows behind the context, in place: for i < num_accepted[s],
 * position context_lens[s] - n_s + accepted[s][i] is copied to position context_lens[s] -
 * n_s + i, K and V of every kv head. Codes of fp8 / int8 caches move as they are between
 * blocks with equal scales (and zero points); otherwise their value is converted again
 * with the destination's, as reshape_and_cache would. Positions behind the path keep what
 * they held. The positions written must lie in blocks that no other sequence shares. A path
 * that is not strictly ascending within the sequence's rows moves nothing (PA_DEVERR_TREE).
 * accepted: int32 [num_seqs][max_accept], max_accept at most 256.
 */
pa_status compact_accepted(void* k_cache, void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, const int32_t* query_start,
                           const int32_t* accepted, const int32_t* num_accepted, int num_seqs,
                           int max_accept, int max_blocks_per_seq, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, pa_dtype cache_dtype,
                           const float* k_scales, const float* v_scales,
                           const int32_t* k_zeros, const int32_t* v_zeros, void* stream);

/*
 * Reads and clears the device error word of the current device (a bitwise OR of
 * PA_DEVERR_* recorded by kernels since the last call). Synchronises `stream` first.
 * Returns PA_OK when the word was 0, PA_ERR_DEVICE otherwise (bits in *bits_out).
 */
pa_status pa_device_error(int* bits_out, void* stream);

/*
 * Selects the decode kernels used by later paged_attn_decode calls in this process:
 * 0 = automatic (tensor cores for bf16 / fp8 / int8 caches where the shape is supported:
 * persistent warp workers for partitions <= 512 tokens, else one CTA per work item; else
 * the CUDA-core fp32 path), 1 = CUDA-core path only, 2 = same as 0, 3 / 4 / 5 = tensor
 * cores with a fixed kernel where the call allows it: 3 one CTA per work item, 4
 * persistent CTAs that share each work item (split path, partitions <= 2048 tokens), 5
 * persistent warp workers, one work item per warp (split path, partitions <= 512 tokens). All compute the
 * same function; they differ in how work is scheduled and how q.K and P.V are multiplied.
 * Returns PA_ERR_INVALID for any other value. Not thread-safe.
 */
pa_status pa_set_decode_impl(int impl);

/* Library version string, e.g. "pagedattn 0.1 sm_100a". */
const char* pa_version(void);

/* ------------------------------------------------------------------------------------- */
/* Host block allocator ([Ch4PA] "Borrowing the fix from OS paging": a free list of       */
/* fixed-size units; [KVFail] Key Points: blocks come from a free queue and an allocation */
/* fails when too few are free; [KVPaged] "Prefix sharing and copy-on-write" and [Ch4PA]  */
/* "Prefix Caching": ref_count per block, copy only on write).                            */
/*                                                                                       */
/* Policy: FIFO free queue (initial order given or 0..N-1); allocation pops the front; a */
/* block whose ref_count reaches 0 is pushed to the back. add_seq allocates              */
/* ceil(n/block_size) blocks; fork copies the parent's table and length and increments  */
/* every block's ref_count; append first copies the last block if it is partially filled */
/* AND shared (one new block, the pair (old, new) reported, old loses one reference),    */
/* then pops one block per new block boundary crossed. Every call either succeeds fully  */
/* or returns an error and changes nothing. Host only; not thread-safe; the caller owns   */
/* the object. Sequence ids are any non-negative int.                                    */
/* ------------------------------------------------------------------------------------- */
typedef struct pa_allocator pa_allocator;

/* NULL on bad sizes / allocation failure. */
pa_allocator* pa_alloc_create(int num_blocks, int block_size);
/* `order`: host int32[num_blocks], a permutation of 0..num_blocks-1 giving the initial
 * free-queue order. NULL when it is not a permutation. */
pa_allocator* pa_alloc_create_ordered(int num_blocks, int block_size, const int32_t* order);
void pa_alloc_destroy(pa_allocator* a);
int pa_alloc_num_free(const pa_allocator* a);
/* -1 for a block id out of range. */
int pa_alloc_ref_count(const pa_allocator* a, int block);
/* New sequence of num_tokens tokens; host int64 slots_out[num_tokens] (may be NULL)
 * receives slot = block*block_size + offset of every token. */
pa_status pa_alloc_add_seq(pa_allocator* a, int seq_id, int num_tokens, int64_t* slots_out);
pa_status pa_alloc_fork(pa_allocator* a, int parent_id, int child_id);
/* Appends num_tokens tokens; slots_out[num_tokens] receives their slots; cow_pairs_out
 * (host int32[2], may be NULL only if no copy can occur) receives (src, dst) of the
 * copy-on-write copy and *num_cow_out is 0 or 1. */
pa_status pa_alloc_append(pa_allocator* a, int seq_id, int num_tokens, int64_t* slots_out,
                          int32_t* cow_pairs_out, int* num_cow_out);
/*
 * One decode step's appends in one call: num_tokens[i] tokens to sequence seq_ids[i] for
 * i = 0 .. n-1, in that order, with the same results as n pa_alloc_append calls, except
 * that the batch is all-or-nothing: when the free queue cannot serve the whole batch (the
 * copies included), PA_ERR_NO_BLOCKS is returned and nothing changes. Sequence ids must be
 * distinct and known (else PA_ERR_INVALID, nothing changed).
 *   seq_ids, num_tokens  host int32 [n]
 *   slots_out            host int64 [sum of num_tokens] or NULL: sequence i's slots follow
 *                        sequence i-1's
 *   cow_pairs_out        host int32 [n][2], NULL only if no copy can occur: the (src, dst)
 *                        copy-on-write pairs in batch order; *num_cow_out (may be NULL)
 *                        receives their number
 * One call per step instead of one per sequence keeps the host's share of a decode step
 * small for large batches.
 */
pa_status pa_alloc_append_batch(pa_allocator* a, int n, const int32_t* seq_ids,
                                const int32_t* num_tokens, int64_t* slots_out,
                                int32_t* cow_pairs_out, int* num_cow_out);
pa_status pa_alloc_free_seq(pa_allocator* a, int seq_id);
/* Copies at most `cap` entries of the sequence's block table into out (host int32) and
 * returns the table's length, or -1 for an unknown sequence. */
int pa_alloc_block_table(const pa_allocator* a, int seq_id, int32_t* out, int cap);
/* Tokens held by the sequence, -1 if unknown. */
int pa_alloc_seq_len(const pa_allocator* a, int seq_id);
/* Writes the free queue front-to-back into out (at most cap entries); returns its size. */
int pa_alloc_free_queue(const pa_allocator* a, int32_t* out, int cap);

/* ------------------------------------------------------------------------------------- */
/* Automatic prefix caching ([Ch4PA] "Prefix Caching": a SHA-256 hash of the prefix       */
/* identifies identical blocks and hits raise ref_count; [KVPaged] "Prefix cache lifetime */
/* and invalidation": a hit skips recomputing the prefix KV, eviction is least recently   */
/* used; [KVFail] Key Points: a cached block is evicted when the free queue hands it out). */
/* Every full block i of a sequence added with its tokens gets the chained hash           */
/*   h_i = SHA-256(h_{i-1} || tokens of block i as little-endian int32), h_{-1} empty.    */
/* ------------------------------------------------------------------------------------- */
/*
 * New sequence of num_tokens token ids (host int32 tokens[num_tokens]). Its longest run of
 * leading full blocks whose hashes are cached is reused (ref_count + 1; a cached block
 * waiting in the free queue is taken out of it); the remaining blocks are popped from the
 * queue front (a popped block loses any cache entry it had: eviction) and its other full
 * blocks are registered in the cache. slots_out[num_tokens] receives every token's slot;
 * *cached_tokens_out (may be NULL) the number of leading tokens whose K/V is already in
 * the cache (the caller writes only the tokens after them). A freed block keeps its entry
 * while it waits in the free queue. PA_ERR_NO_BLOCKS (nothing changed) when the free queue,
 * minus the cached blocks this call reuses, is too short.
 */
pa_status pa_alloc_add_seq_tokens(pa_allocator* a, int seq_id, const int32_t* tokens,
                                  int num_tokens, int64_t* slots_out, int* cached_tokens_out);
/* Number of blocks with a prefix-cache entry (in use or waiting in the free queue). */
int pa_alloc_num_cached(const pa_allocator* a);
/* Totals since creation: blocks reused by hits, cache entries evicted. */
pa_status pa_alloc_cache_stats(const pa_allocator* a, int64_t* hit_blocks, int64_t* evictions);
/* Copies block's chained hash (32 bytes) into out32 and returns 1, or returns 0 when the
 * block has no cache entry. */
int pa_alloc_block_hash(const pa_allocator* a, int block, uint8_t* out32);
/* SHA-256 (FIPS 180-4) of len bytes at data into out32: the hash the prefix cache uses. */
void pa_sha256(const void* data, size_t len, uint8_t* out32);

#ifdef __cplusplus
}
#endif
#endif /* PAGEDATTN_H_ */
