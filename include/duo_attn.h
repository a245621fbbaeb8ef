/*
 * duo_attn.h -- C ABI of a GB300 (sm_103a) library for mixed-head causal attention
 * in long-context serving: retrieval heads over a full KV cache, streaming heads
 * over a sink + ring-buffer cache.
 *
 * What the operations compute (sources are the pages this library restates):
 *
 *   DuoAttention README (mit-han-lab/duo-attention), Abstract: a few attention heads
 *   ("retrieval heads") need full attention over every token and keep a full KV
 *   cache; the others ("streaming heads") look mostly at the attention sinks and
 *   the recent tokens and keep a constant-size cache. With S = sink_size and
 *   R = recent_size (quick start: S = 64, R = 256), query position i of a head sees
 *   key position j when
 *       retrieval:  j <= i
 *       streaming:  j <= i  and  (j < S  or  i - j < R)
 *   and the output is softmax(q.k / sqrt(head_dim)) over the visible keys, times v.
 *
 *   vLLM issue "Could you support Attention Sink?", block tables and its option 3:
 *   sink tokens stay in their own slots and later tokens wrap around a circular
 *   buffer, so nothing is ever moved. Token t is stored in slot t if t < S, else in
 *   slot S + ((t - S) mod R).
 *
 *   transformers pull request "[WIP] Dynamic length in static cache": a decode step
 *   attends only to the positions written so far, never to the unused capacity.
 *
 * Conventions for every call:
 *   - All tensors are caller-owned device memory (e.g. torch tensors); the library
 *     allocates no device memory and never synchronises the device, except in
 *     duo_device_error().
 *   - bf16 means IEEE-754 binary16 "brain float" (torch.bfloat16). Tensors are dense
 *     and row-major in the index order written; base addresses must be 16-byte
 *     aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Every kernel runs on it, asynchronously to the host. The append and decode
 *     kernels, those of the 8-bit caches and of the block tables use programmatic dependent
 *     launch among themselves (an append lets the decode after it start early, each waits
 *     for the grid before it before touching its data); stream order holds as usual for any
 *     kernel launched without the cudaLaunchAttributeProgrammaticStreamSerialization
 *     attribute. A caller kernel launched with that attribute right after one of them must
 *     call cudaGridDependencySynchronize() before it reads what they wrote.
 *   - Arguments are checked on the host before any launch. On an error nothing is
 *     written, the cache length is unchanged, the status is returned and
 *     duo_last_error() describes it.
 *   - A handle holds host state only; it may be used from one host thread at a
 *     time. The device is the one current when duo_create ran.
 */
#ifndef DUO_ATTN_H_
#define DUO_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DUO_OK = 0,
  DUO_ERR_INVALID_ARG = 1,    /* null pointer, bad size, misaligned address */
  DUO_ERR_UNSUPPORTED = 2,    /* a shape the kernels do not implement (see duo_config) */
  DUO_ERR_CAPACITY = 3,       /* the append would exceed max_seq_len */
  DUO_ERR_CUDA = 4,           /* a CUDA runtime or driver call failed (launch error) */
  DUO_ERR_DEVICE_TIMEOUT = 5, /* a kernel gave up a bounded wait (see duo_device_error) */
  DUO_ERR_WORKSPACE = 6       /* decode workspace missing or smaller than required */
} duo_status;

/* Head kinds, one per KV head. A query head h uses KV head h / (num_q_heads /
 * num_kv_heads) and inherits its kind. */
#define DUO_STREAMING 0
#define DUO_RETRIEVAL 1

typedef struct {
  int32_t batch;        /* B >= 1 */
  int32_t num_q_heads;  /* Hq, a multiple of num_kv_heads, Hq / Hkv in {1, 2, 4, 8} */
  int32_t num_kv_heads; /* Hkv, 1 ... 128 */
  int32_t head_dim;     /* D in {64, 128} */
  int32_t sink_size;    /* S >= 0 */
  int32_t recent_size;  /* R >= 1 (R = 0 would leave a query with no key) */
  int64_t max_seq_len;  /* capacity of each retrieval head's cache, in tokens */
} duo_config;

typedef struct duo_handle duo_handle;

/* The caches of one layer. All pointers are device pointers owned by the caller.
 *   k_full, v_full : bf16 [B, n_ret, max_seq_len, D]; row t of retrieval head r holds
 *                    token t for t < n. Rows >= n are never read.
 *   k_sr, v_sr     : bf16 [B, n_str, S + R, D]; the sink slots then the ring slots of
 *                    each streaming head.
 *   pos            : int32 [B, S + R]; the token position held by each slot, -1 if
 *                    empty. Shared by all streaming heads of a sequence.
 *   n              : tokens appended so far (the same for every sequence of the batch).
 * n_ret / n_str are the numbers of retrieval / streaming KV heads; a pointer whose
 * count is zero may be NULL. The compact order of heads of one kind is increasing
 * KV-head index (see duo_classify_heads). Initialise a cache with duo_cache_reset. */
typedef struct {
  void* k_full;
  void* v_full;
  void* k_sr;
  void* v_sr;
  int32_t* pos;
  int64_t n;
} duo_kv_cache;

/* Per-head retrieval/streaming mask (host only, no device work).
 * is_retrieval[Hkv]: nonzero = retrieval. Writes kind_index[h] = the index of KV head
 * h among the heads of its kind (its plane in k_full/v_full or k_sr/v_sr), and
 * *n_retrieval. Source: the DuoAttention README's quick start turns trained per-head
 * gate values into a binary retrieval/streaming choice per head. */
duo_status duo_classify_heads(const uint8_t* is_retrieval, int32_t num_kv_heads, int32_t* kind_index,
                              int32_t* n_retrieval);

/* Create a handle for one layer shape and head mask (host arrays, copied). */
duo_status duo_create(const duo_config* config, const uint8_t* is_retrieval, duo_handle** out);
void duo_destroy(duo_handle* handle);

/* Re-classify the KV heads of an existing handle (host array of num_kv_heads flags,
 * copied), e.g. after loading another head pattern. The caches are laid out by kind
 * ([B, n_ret, ...] and [B, n_str, ...]), so the caller must re-lay them out (or reset
 * and refill them) for the new counts before the next call that uses them; the shape
 * of the handle is otherwise unchanged. The DuoAttention README's patch applies a
 * loaded head pattern the same way: one mask per layer. */
duo_status duo_set_head_mask(duo_handle* handle, const uint8_t* is_retrieval);

/* Empty the cache: pos[] := -1 on `stream`, cache->n := 0. */
duo_status duo_cache_reset(duo_handle* handle, duo_kv_cache* cache, void* stream);

/* Append T >= 1 new tokens at positions n ... n+T-1 and set cache->n += T.
 * k_new, v_new: bf16 [B, T, Hkv, D] (token-major, as a fused QKV projection emits).
 * Retrieval heads: rows n ... n+T-1 of k_full/v_full. Streaming heads: each token goes
 * to slot t (t < S) or S + ((t - S) mod R); of the tokens of one call only those still
 * held when the call ends are written (t < S, or t >= n+T-R), so the result equals T
 * single-token appends and no slot is written twice. pos[] is updated to match.
 * DUO_ERR_CAPACITY if n + T > max_seq_len (nothing written). */
duo_status duo_kv_append(duo_handle* handle, duo_kv_cache* cache, const void* k_new, const void* v_new, int32_t T,
                         void* stream);

/* Prefill attention of T >= 1 new tokens at positions n ... n+T-1 (n = cache->n, the
 * cache state BEFORE these tokens are appended; n = 0 for a one-shot prefill, n > 0
 * for a chunk of a chunked prefill against the growing cache).
 * q: bf16 [B, T, Hq, D]; k, v: bf16 [B, T, Hkv, D] of the same tokens; o: bf16
 * [B, T, Hq, D]. A retrieval head attends to cache rows [0, n) and to the new tokens;
 * a streaming head to what its sink + ring cache holds and to the new tokens, each
 * with the visibility rule above. Scale 1/sqrt(D) is applied in fp32 to the fp32
 * product; softmax and accumulation are fp32; o is rounded to nearest even.
 * The cache is not modified: call duo_kv_append(k, v) afterwards.
 * Fully masked key tiles are skipped, so a streaming head costs O((S + R) * T). */
duo_status duo_attn_prefill(duo_handle* handle, const duo_kv_cache* cache, const void* q, const void* k,
                            const void* v, int32_t T, void* o, void* stream);

/* As duo_attn_prefill, restricted to the query heads whose KV head kind bit is set in
 * kind_mask (bit 0 = streaming, bit 1 = retrieval). Rows of o for other heads are not
 * written. Used to time the retrieval heads alone. */
duo_status duo_attn_prefill_select(duo_handle* handle, const duo_kv_cache* cache, const void* q, const void* k,
                                   const void* v, int32_t T, void* o, int32_t kind_mask, void* stream);

/* Bytes of device workspace the decode entry points (duo_attn_decode, _paged, _varlen,
 * duo_dca_decode, duo_attn_decode_kv4, duo_attn_decode_kv8) need for a cache of n tokens; the size covers
 * the largest grid any of them launches, so one workspace serves them all. */
size_t duo_decode_workspace_size(const duo_handle* handle, int64_t n);

/* One decode step for the token at position p = cache->n - 1, which must already have
 * been appended (duo_kv_append with T = 1). q: bf16 [B, Hq, D]; o: bf16 [B, Hq, D].
 * Reads rows [0, n) of each retrieval head and the valid slots of each streaming head
 * (each slot checked against pos[] and the visibility rule), every K/V byte once per
 * KV head for all its query heads. The keys are split over the GPU's SMs; partial
 * softmaxes (o, max, sum) go to `workspace` and are merged by log-sum-exp.
 * workspace: device memory of at least duo_decode_workspace_size(handle, n) bytes,
 * 256-byte aligned. It holds the partial softmax results (o, max, sum) of the
 * (sequence, KV head) pairs split over several CTAs, which a second kernel merges
 * right after the decode kernel (its programmatic dependent); nothing in it has to
 * survive between calls, so the memory may hold anything between calls.
 * Calls sharing one workspace must be ordered on the GPU (same stream). */
duo_status duo_attn_decode(duo_handle* handle, const duo_kv_cache* cache, const void* q, void* o, void* workspace,
                           size_t workspace_bytes, void* stream);

/* duo_attn_decode without a workspace argument, for callers that cannot allocate
 * device memory for scratch (an engine that has handed all device memory to its own
 * pool, a loop that must not call cudaMalloc/cudaFree because they may synchronise,
 * a runtime whose allocator owns every allocation). The pages have no counterpart:
 * it is an interface variant of the decode step above and computes the same result.
 * Scratch lives in a 2 MiB array inside the library (every GPU that loads the library
 * holds it until the process exits); shapes whose bf16 decode scratch (one partial
 * of g (D + 4) floats per CTA and per (sequence, KV head), with one CTA per SM)
 * exceeds 2 MiB get DUO_ERR_WORKSPACE. Nothing is
 * allocated: no cudaMalloc, cudaFree or allocating library call. The first call on
 * each device, and the first in any other CUDA context made current there later (after
 * cudaDeviceReset, say), looks up the array's device address (cudaGetSymbolAddress);
 * make that first call before any stream capture. All calls on a device share the
 * one array, so calls that overlap on the GPU (different streams, or several host
 * threads) race: order them on one stream. */
duo_status duo_attn_decode_static(duo_handle* handle, const duo_kv_cache* cache, const void* q, void* o,
                                  void* stream);

/* Paged caches, as a block allocator hands out memory in a serving engine (vLLM issue
 * "Could you support Attention Sink?" discusses the cache as fixed-size token blocks
 * chained by a block table, and keeping the first block as the sinks while dropping
 * the middle blocks and keeping the recent ones). With a duo_paged descriptor,
 * cache->k_full and cache->v_full are pools of blocks, bf16 [num_blocks, block_size,
 * D], shared by every sequence and head; row t of retrieval head r of sequence b is
 * row t % block_size of block block_table[(b * n_ret + r) * max_blocks + t / block_size].
 *
 * stream_table == NULL: streaming heads keep their sink + ring cache (cache->k_sr,
 * v_sr, pos). stream_table != NULL: streaming heads live in the same pools too, token
 * t of streaming head s of sequence b at row t % block_size of block
 * stream_table[(b * n_str + s) * max_blocks + t / block_size]; cache->k_sr, v_sr and pos
 * are then not used (may be NULL). Block granularity is only a storage choice: a query
 * still sees exactly the sinks and its recent window, token by token, so results match
 * the ring cache up to fp32 summation order. Once the cache holds n tokens, the blocks
 * duo_paged_stream_dead_blocks names hold no token any later query can see: the caller
 * may free them (their table entries are never read again). An append writes a
 * streaming token only if its block is still live when the call ends, so only live
 * blocks need to exist: the sink blocks and those reaching back R tokens from the end.
 *
 * The capacity of a head is block_size * max_blocks tokens (max_seq_len is not used).
 * A block id outside [0, num_blocks) that would be read or written is never
 * dereferenced: its rows are skipped and duo_device_error() reports
 * DUO_ERR_INVALID_ARG (a prefill over bf16 pools reads them as zeros, which take part in its
 * softmax; decodes and the 8-bit prefill leave them out). Other rows, and later calls, are
 * not affected. Retrieval results equal the contiguous layout's, bit for bit. */
typedef struct {
  const int32_t* block_table;  /* int32 [B, n_ret, max_blocks], device memory (NULL if n_ret = 0) */
  int32_t block_size;          /* rows per block, a positive multiple of 128 */
  int32_t max_blocks;          /* table entries per (sequence, head) */
  int64_t num_blocks;          /* blocks in each pool */
  const int32_t* stream_table; /* int32 [B, n_str, max_blocks], device memory, or NULL */
} duo_paged;

/* Logical blocks [*lo, *hi) of a paged streaming head that no query at a position
 * >= n - 1 can see once the cache holds n tokens: blocks past the sink blocks
 * (lo = ceil(S / block_size)) that end at or before the recent window of the last
 * token (hi = max(lo, floor(max(0, n - R) / block_size))). The range only grows with
 * n, so after each call the caller may free [previous hi, hi). Host only. */
duo_status duo_paged_stream_dead_blocks(int32_t sink_size, int32_t recent_size, int32_t block_size, int64_t n,
                                        int64_t* lo, int64_t* hi);

duo_status duo_kv_append_paged(duo_handle* handle, duo_kv_cache* cache, const duo_paged* paged, const void* k_new,
                               const void* v_new, int32_t T, void* stream);
duo_status duo_attn_prefill_paged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                  const void* q, const void* k, const void* v, int32_t T, void* o, void* stream);
duo_status duo_attn_decode_paged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                 const void* q, void* o, void* workspace, size_t workspace_bytes, void* stream);

/* 4-bit KV caches. The DuoAttention README pairs the method with a 4-bit KV cache to
 * decode millions of tokens on one GPU (quick-start demo, Efficiency section) but gives
 * no format; this library uses the plainest asymmetric one. Each cached row (the D
 * values of one token of one head) is stored as D 4-bit codes plus an fp16 scale and
 * zero: scale = fp16((max - min) / 15), zero = fp16(min), code = clamp(rint((x - zero)
 * / scale), 0, 15) with every step in fp32 round-to-nearest (all codes 0 when the
 * scale is 0), value = code * scale + zero. Codes are packed two per byte, the even
 * dim in the low nibble. Rows must stay within the fp16 range.
 *
 * K codes are stored row by row (D / 2 bytes per row). V codes are stored in groups of
 * 16 rows (rows 16 m ... 16 m + 15 of a plane, 8 D bytes), ordered for the decode's
 * tensor-core fragments: the byte with the codes of dims 2 dp (low nibble) and 2 dp + 1
 * (high nibble) of row k of the group sits at byte
 *     4 ((4 (dp / MT) + (k % 8) / 2) MT + dp % MT) + 2 (k % 2) + k / 8,   MT = D / 16,
 * of the group. Each byte belongs to one row, so appending a row writes only its bytes.
 *
 * Layout (all device memory, caller-owned, 16-byte aligned), with cap16 = max_seq_len
 * and sr16 = S + R each rounded up to a multiple of 16 rows:
 *   k_codes, v_codes    u8  [B, n_ret, cap16, D / 2]   retrieval heads, row t = token t
 *   k_sz, v_sz          u32 [B, n_ret, cap16]          fp16 scale (low half), zero (high)
 *   ks_codes, vs_codes  u8  [B, n_str, sr16, D / 2]    streaming heads, sink + ring slots
 *   ks_sz, vs_sz        u32 [B, n_str, sr16]
 * cache->n and cache->pos keep their meaning; cache->k_full, v_full, k_sr, v_sr are not
 * used. duo_kv_append_kv4 quantizes and stores the new tokens (same slot rule as
 * duo_kv_append); duo_attn_decode_kv4 is duo_attn_decode over these arrays, with the
 * dequantization folded into the dot products (q . k = scale (q . codes) + zero sum(q)).
 * duo_attn_prefill_kv4 prefills a chunk against caches in this form.
 *
 * duo_attn_decode_kv4 runs its dot products on the tensor cores with fp16 operands
 * (codes, q, and p times the row scale, stored as p scale / 64) and fp32 accumulation,
 * so q must lie within the fp16 range as well (bf16 values there convert exactly).
 * Its workspace is the one duo_decode_workspace_size gives; it launches two CTAs per
 * SM. Errors: as duo_attn_decode, plus DUO_ERR_INVALID_ARG for a NULL or misaligned
 * array the handle's head kinds need (every array 16-byte aligned). */
typedef struct {
  void* k_codes;
  void* v_codes;
  void* k_sz;
  void* v_sz;
  void* ks_codes;
  void* vs_codes;
  void* ks_sz;
  void* vs_sz;
} duo_kv4_cache;

duo_status duo_kv_append_kv4(duo_handle* handle, duo_kv_cache* cache, const duo_kv4_cache* kv4, const void* k_new,
                             const void* v_new, int32_t T, void* stream);
duo_status duo_attn_decode_kv4(duo_handle* handle, const duo_kv_cache* cache, const duo_kv4_cache* kv4,
                               const void* q, void* o, void* workspace, size_t workspace_bytes, void* stream);

/* Prefill of T new tokens against 4-bit caches (chunked prefill after earlier chunks were
 * appended with duo_kv_append_kv4): as duo_attn_prefill, with the keys and values of the
 * cache rows (retrieval rows [0, n), valid sink + ring slots) read from `kv4` and
 * dequantized (code * scale + zero in fp32, rounded to bf16) into the kernel's shared-memory
 * tiles, so no bf16 copy of the cache exists anywhere; the T new tokens' k and v are the bf16
 * inputs as usual. Append the chunk afterwards with duo_kv_append_kv4. cache->k_full,
 * v_full, k_sr, v_sr are not used. Errors: as duo_attn_prefill, plus those of the 4-bit
 * arrays (see duo_attn_decode_kv4). */
duo_status duo_attn_prefill_kv4(duo_handle* handle, const duo_kv_cache* cache, const duo_kv4_cache* kv4,
                                const void* q, const void* k, const void* v, int32_t T, void* o, void* stream);

/* 4-bit caches with the retrieval rows in a paged pool (the two layouts above combined:
 * the block allocator of the attention-sink issue holding the 4-bit rows the README
 * pairs the method with). kv4->k_codes, v_codes are pools u8 [num_blocks, block_size,
 * D / 2] and kv4->k_sz, v_sz pools u32 [num_blocks, block_size]; row t of retrieval head
 * r of sequence b is row t % block_size of block paged->block_table[(b n_ret + r)
 * max_blocks + t / block_size] (block_size a multiple of 128, so 16-row V groups never
 * straddle blocks). The row encoding and the V group order are those of the contiguous
 * 4-bit arrays. Streaming heads keep their 4-bit sink + ring arrays: paged->stream_table
 * must be NULL (DUO_ERR_UNSUPPORTED otherwise). Capacity, bad block ids and errors: as
 * duo_kv_append_paged / duo_attn_decode_paged (a bad id is reported by duo_device_error,
 * its rows are neither written nor read). */
duo_status duo_kv_append_kv4_paged(duo_handle* handle, duo_kv_cache* cache, const duo_paged* paged,
                                   const duo_kv4_cache* kv4, const void* k_new, const void* v_new, int32_t T,
                                   void* stream);
duo_status duo_attn_decode_kv4_paged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                     const duo_kv4_cache* kv4, const void* q, void* o, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* 8-bit KV caches: the retrieval heads' rows as 8-bit codes, with one fp32 scale for each
 * block of DUO_KV8_BLOCK = 64 tokens of one head (K and V apart). Half the bytes of the
 * bf16 caches at decode, and a milder rounding than the 4-bit ones. Streaming heads keep
 * their bf16 sink + ring caches (cache->k_sr, v_sr, pos), whose size does not grow.
 *
 * Tokens 64 j ... 64 j + 63 of a head form block j. When the block is full its rows are
 * rounded, once, from their bf16 values x:
 *     DUO_KV8_INT8:  scale = fp32(amax / 127),  code = clamp(rint(fp32(x / scale)), -127, 127)
 *     DUO_KV8_E4M3:  scale = fp32(amax / 448),  code = e4m3(fp32(x / scale)), saturating
 * amax = the largest |x| of the block's 64 x D values, every step rounded to nearest even;
 * value = code * scale. A block of zeros has scale 0 and codes 0; a block with an infinity
 * or a NaN has scale NaN and codes 0 (its head's outputs are then NaN, never silently wrong).
 * The rows of the block that is not full yet stay in bf16, in the tail: row t of the open
 * block at row t % 64 of the (sequence, head)'s tail. So T appends of one token leave the
 * same cache as one append of T, and recent tokens are exact.
 *
 * Layout (device memory, caller-owned, 16-byte aligned), cap64 = max_seq_len rounded up to
 * a multiple of 64:
 *   k_codes, v_codes  8-bit [B, n_ret, cap64, D]     row t = token t
 *   k_scale, v_scale  fp32  [B, n_ret, cap64 / 64]
 *   k_tail, v_tail    bf16  [B, n_ret, 64, D]
 * With a duo_paged descriptor (the _paged, _ragged and _varlen entry points;
 * paged->stream_table must be NULL) the codes and scales are pools:
 *   k_codes, v_codes  8-bit [num_blocks, block_size, D]     (rows addressed as in duo_paged)
 *   k_scale, v_scale  fp32  [num_blocks, block_size / 64]
 * cache->n and cache->pos keep their meaning; cache->k_full and v_full are not used. Every
 * pointer may be NULL when the handle has no retrieval head. The rows of the codes (B n_ret
 * cap64, or num_blocks block_size) must stay below 2^31. */
#define DUO_KV8_BLOCK 64
#define DUO_KV8_INT8 0
#define DUO_KV8_E4M3 1

typedef struct {
  void* k_codes;
  void* v_codes;
  float* k_scale;
  float* v_scale;
  void* k_tail;
  void* v_tail;
  int32_t code_type; /* DUO_KV8_INT8 or DUO_KV8_E4M3 */
} duo_kv8_cache;

/* duo_kv_append into these caches: T new tokens at positions n ... n+T-1 (k_new, v_new:
 * bf16 [B, T, Hkv, D]). Full blocks are written as codes, the open block's rows to the
 * tail; everything else of the arrays is left as it was. Capacity and errors as
 * duo_kv_append / duo_kv_append_paged. */
duo_status duo_kv_append_kv8(duo_handle* handle, duo_kv_cache* cache, const duo_kv8_cache* kv8, const void* k_new,
                             const void* v_new, int32_t T, void* stream);
duo_status duo_kv_append_kv8_paged(duo_handle* handle, duo_kv_cache* cache, const duo_paged* paged,
                                   const duo_kv8_cache* kv8, const void* k_new, const void* v_new, int32_t T,
                                   void* stream);

/* Where the tokens of a packed batch go (device memory; duo_block_tables_update writes it):
 *   cu_new    int32 [B + 1]             tokens cu_new[b] ... cu_new[b + 1] - 1 are sequence b's
 *   token_seq int32 [num_tokens]        the sequence of each token, -1 for padding
 *   token_pos int32 [num_tokens]        its position in the sequence, -1: not stored
 *   slots     int64 [num_tokens, n_ret] its row in the pool for each retrieval head (block id
 *                                       times block_size plus the row in the block), -1: none
 * Tokens of one sequence follow each other at consecutive positions, and a sequence has its
 * tokens in one piece. */
typedef struct {
  int32_t* cu_new;
  int32_t* token_seq;
  int32_t* token_pos;
  int64_t* slots;
} duo_slot_map;

/* Append of a packed batch, each sequence with its own length and number of new tokens:
 * k_new, v_new: bf16 [num_tokens, Hkv, D], 0 <= num_tokens. The positions and rows come from
 * `map` alone (cache->n is neither read nor changed, no table is read), so a step captured
 * in a CUDA graph replays with other lengths. Tokens at position -1 are skipped and nothing
 * of their sequence changes. A slot or sequence out of range is not dereferenced: its rows
 * are skipped and duo_device_error() reports DUO_ERR_INVALID_ARG; so it is with the tokens of a
 * sequence whose last position would reach 2^31 - 1. */
duo_status duo_kv_append_kv8_ragged(duo_handle* handle, duo_kv_cache* cache, const duo_paged* paged,
                                    const duo_kv8_cache* kv8, const duo_slot_map* map, int32_t num_tokens,
                                    const void* k_new, const void* v_new, void* stream);

/* One decode step over 8-bit caches, as duo_attn_decode (same q, o, workspace and order of
 * calls): scores and outputs are accumulated in fp32 from the codes (fp16 tensor-core
 * operands, exact for both code types; q scaled to fp16 by a power of two of its own per
 * head, so any finite bf16 q is taken) and the tail and ring rows (bf16 operands); p is
 * rounded to fp16 over codes and to two bf16 terms (2^-17) over bf16 rows. Workspace as for
 * duo_attn_decode; o must not overlap q.
 * duo_attn_decode_kv8_varlen reads the lengths on the device (seq_lens int32 [B], clamped
 * to [0, max_len], the new token included; a sequence of length 0 gets zeros) and splits the
 * work by them; `paged` may be NULL (contiguous caches). */
duo_status duo_attn_decode_kv8(duo_handle* handle, const duo_kv_cache* cache, const duo_kv8_cache* kv8, const void* q,
                               void* o, void* workspace, size_t workspace_bytes, void* stream);
duo_status duo_attn_decode_kv8_paged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                     const duo_kv8_cache* kv8, const void* q, void* o, void* workspace,
                                     size_t workspace_bytes, void* stream);
duo_status duo_attn_decode_kv8_varlen(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                      const duo_kv8_cache* kv8, const int32_t* seq_lens, int64_t max_len,
                                      const void* q, void* o, void* workspace, size_t workspace_bytes, void* stream);

/* Prefill of T new tokens against 8-bit caches, as duo_attn_prefill: the cache's rows are
 * code * scale (tail and ring rows are bf16), the T new tokens' k and v the bf16 inputs.
 * Append the chunk afterwards. Every sequence holds cache->n tokens and takes T: there is no form
 * with lengths on the device, so ragged prompts are prefilled a sequence (or a group of one length)
 * at a time, through a handle of that batch. The codes are written to `workspace` once, as bf16 times the
 * power of two in their scale (exact; the rest of the scale is applied in fp32, V's to p before
 * p is rounded to bf16), and read from there by every query block; retrieval heads with few
 * query blocks are split over their keys, their parts merged by log-sum-exp. workspace:
 * device memory of duo_prefill_kv8_workspace_size(handle, cache->n, T) bytes, 256-byte
 * aligned (may be NULL if that is 0: nothing cached, or no retrieval head): 4 D bytes per
 * cached token and retrieval head of the layer, 8 per 64 of them, plus the parts (at most 8 per SM, and none when
 * the split would not pay, so a longer cache can need less: ask for each n and T). Nothing in it
 * survives the call; calls sharing one must be ordered on the GPU. o must not overlap q, k or v. */
size_t duo_prefill_kv8_workspace_size(const duo_handle* handle, int64_t n, int32_t T);
duo_status duo_attn_prefill_kv8(duo_handle* handle, const duo_kv_cache* cache, const duo_kv8_cache* kv8,
                                const void* q, const void* k, const void* v, int32_t T, void* o, void* workspace,
                                size_t workspace_bytes, void* stream);
duo_status duo_attn_prefill_kv8_paged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                      const duo_kv8_cache* kv8, const void* q, const void* k, const void* v,
                                      int32_t T, void* o, void* workspace, size_t workspace_bytes, void* stream);

/* Block tables kept on the device. A pool of num_blocks blocks of block_size tokens serves
 * B sequences with `planes` tables each (planes = n_ret: one per retrieval head).
 *   block_table int32 [B, planes, max_blocks]  entry j of a plane: the block of its tokens
 *                                              block_size j ...; entries past the length are
 *                                              not read
 *   free_list   int32 [num_blocks]             ids of the free blocks: the first *free_count
 *   free_count  int32 [1]
 *   seq_lens    int32 [B]                      tokens each sequence holds
 * all device memory. B planes max_blocks and block_size max_blocks must stay below 2^31. */
typedef struct {
  int32_t* block_table;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* seq_lens;
  int32_t batch;
  int32_t planes;
  int32_t block_size; /* >= 1; a multiple of 128 for the attention entry points */
  int32_t max_blocks;
  int64_t num_blocks;
} duo_block_pool;

/* Brings tables, free list and lengths up to date for a step in which sequence b takes
 * new_lens[b] >= 0 more tokens, or has finished (new_lens[b] = -1), and writes the slot map
 * of the packed new tokens (arrays of max_tokens tokens). All on the device, so the call can
 * be captured in a CUDA graph and replayed. In this order:
 *   1. Finished sequences, by index: the blocks of their planes (plane by plane, first block
 *      first) go onto the end of the free list; their length becomes 0. Their table entries
 *      are left as they are.
 *   2. The others, by index: a sequence that needs new blocks gets them if the free list
 *      holds enough for it and all sequences before it; otherwise neither it nor any later
 *      one that needs blocks gets any. Blocks are taken from the end of the free list, for
 *      plane 0 first. A sequence is also turned down if it would pass max_blocks or if its
 *      tokens pass max_tokens. A sequence that was turned down keeps its length, its tokens
 *      get position and slots -1, and duo_device_error() reports DUO_ERR_CAPACITY.
 * cu_new[b] is the sum of max(new_lens, 0) of the sequences before b, served or not (up to
 * 2^31 - 1). Tokens past cu_new[B] are padding: sequence, position and slots -1.
 * seq_lens_out [B] and free_count_out [1] receive the new lengths and count; they may be
 * pool->seq_lens and pool->free_count. If they are not, the call leaves both inputs as they
 * were, and the same call again gives the same result.
 * A length below 0 or past the tables, new_lens below -1, a free count outside [0,
 * num_blocks] (clamped) or a block id outside [0, num_blocks) (dropped from the free list,
 * slots -1) is reported by duo_device_error() as DUO_ERR_INVALID_ARG; that sequence is
 * turned down. workspace: duo_block_tables_workspace_size(batch) bytes of device memory, 16-byte
 * aligned; nothing in it survives the call, and calls sharing it must be ordered. */
size_t duo_block_tables_workspace_size(int32_t batch);
duo_status duo_block_tables_update(const duo_block_pool* pool, const int32_t* new_lens, int32_t max_tokens,
                                   int32_t* seq_lens_out, int32_t* free_count_out, const duo_slot_map* map,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* A packed ragged step over bf16 paged caches: the tokens of all sequences lie one behind the
 * other, a duo_slot_map says whose they are and where they go, and every length is read on the
 * device, so the calls of a step can be captured in a CUDA graph. In this order:
 *   a step with chunks:  duo_rope_rotate (q, k), duo_attn_prefill_ragged, duo_kv_append_ragged
 *                        (without a rotation: k is rotated already)
 *   one token each:      duo_kv_append_ragged (with the rotation, q beside k),
 *                        duo_attn_decode_paged_varlen
 * Rows are bf16 [num_tokens, heads, D] whose tokens may lie apart, as slices of a fused
 * projection's output do: token t begins x_stride elements after token t - 1 (a multiple of 8,
 * at least heads x D; addresses 16-byte aligned). */
/* Rotary positions. Pair i (0 <= i < rotary_dim / 2) of a row, (a, b), at position p becomes
 *     (scale (a cos t - b sin t), scale (b cos t + a sin t)),  t = p f_i,
 * computed in fp32 from bf16 values and rounded once. The pairs are dims (i, i + rotary_dim / 2)
 * (DUO_ROPE_HALF) or (2 i, 2 i + 1) (DUO_ROPE_INTERLEAVED) of the head; dims from rotary_dim on
 * pass through unchanged. Any frequencies up to 2^40 radians a position will do (scaled ones for long
 * contexts are made on the host); `scale` is the factor that some of these schemes apply to rotated pairs, else 1.
 *   turns: device memory, [rotary_dim / 2], from duo_rope_turns: the angle per position of each
 *          pair as a fraction of a full turn, in units of 2^-64. A position times it wraps as
 *          angles do, so the angle is exact at every position up to 2^31 - 1. */
#define DUO_ROPE_HALF 0
#define DUO_ROPE_INTERLEAVED 1

typedef struct {
  const uint64_t* turns;
  int32_t rotary_dim; /* a multiple of 16, 16 ... head_dim */
  int32_t layout;     /* DUO_ROPE_HALF or DUO_ROPE_INTERLEAVED */
  float scale;
} duo_rope;

/* turns[i] of angles per position inv_freq[i] (radians, up to 2^40 in size), each within one unit. Host
 * arrays; host only. */
duo_status duo_rope_turns(const double* inv_freq, int32_t count, uint64_t* turns);

/* Rotates the rows of q and, unless k is NULL, of k (head_dim 64 or 128) by positions [num_tokens]
 * (int32, device memory); a token at a position below 0 is skipped, its rows of q_out and k_out are
 * left as they were. q_out may be q (with its stride) and k_out k; other overlaps are not allowed. */
duo_status duo_rope_rotate(const duo_rope* rope, int32_t head_dim, const int32_t* positions, int32_t num_tokens,
                           const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                           const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int32_t num_kv_heads,
                           void* stream);

/* Append of a packed batch into bf16 paged caches, each sequence with its own length and number of
 * new tokens: k_new, v_new [num_tokens, Hkv, D]. Positions and rows come from `map` alone, as for
 * duo_kv_append_kv8_ragged: retrieval rows to the pool's rows map->slots, streaming heads' rows to
 * their sink + ring slots (of the tokens of one call only those still held when it ends); tokens at
 * position -1 are skipped; a slot or sequence out of range is not dereferenced, its rows are skipped
 * and duo_device_error() reports DUO_ERR_INVALID_ARG. paged->stream_table must be NULL. cache->n is
 * neither read nor changed. With `rope` (or NULL: none) K is rotated by map->token_pos on the way,
 * and with q and q_out [num_tokens, Hq, D] (or both NULL) q is rotated beside it (q_out may be q). */
duo_status duo_kv_append_ragged(duo_handle* handle, duo_kv_cache* cache, const duo_paged* paged,
                                const duo_slot_map* map, int32_t num_tokens, const duo_rope* rope,
                                const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                                const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, void* stream);

/* Attention of a packed batch of chunks over bf16 paged caches: sequence b's tokens are map->cu_new[b]
 * ... map->cu_new[b + 1] - 1, at the positions from map->token_pos of the first one on, which is also how
 * many tokens its caches hold (before these are appended). q, k, v [num_tokens, Hq or Hkv, D], rotated
 * already; o bf16 [num_tokens, Hq, D], dense. What a query sees is as for duo_attn_prefill: its cached
 * rows (retrieval heads through paged->block_table, streaming heads in cache->k_sr, v_sr, pos) and its
 * own sequence's new tokens; any mixture of single tokens and long chunks may come in one call. A sequence
 * whose first token is at position -1 is skipped, its rows of o and those of padding are left as they
 * were. Scores, softmax and outputs are accumulated in fp32, p is rounded to bf16 before its product
 * with v (to two bf16 terms for a sequence of up to 8 / g tokens).
 * Nothing behind a sequence's last row takes part, whatever it holds (other sequences, padding, rows of a
 * block not written yet); within a sequence, an infinity or NaN in v also reaches queries that do not see
 * it but read its tile of 128 keys.
 * Rows of a block id outside [0, num_blocks) are left out and duo_device_error() reports
 * DUO_ERR_INVALID_ARG; so it does where cu_new falls or passes num_tokens, or a position passes the tables'
 * capacity: that sequence is skipped. paged->stream_table must be NULL.
 * workspace: duo_prefill_ragged_workspace_size(handle, num_tokens) bytes of device memory, 256-byte aligned
 * (parts of items that several CTAs share); nothing in it survives the call, and calls sharing it must be
 * ordered on the GPU. o must not overlap q, k or v. */
size_t duo_prefill_ragged_workspace_size(const duo_handle* handle, int32_t num_tokens);
duo_status duo_attn_prefill_ragged(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                   const duo_slot_map* map, int32_t num_tokens, const void* q, int64_t q_stride,
                                   const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* o,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* Its form for one token a sequence, appended before (as duo_attn_decode): sequence b holds seq_lens[b]
 * tokens (device int32 [B], clamped to [0, max_len], the new one included), its query is at position
 * seq_lens[b] - 1, and a sequence of length 0 gets zeros. q, o: bf16 [B, Hq, D]. Bad block ids as above;
 * a query all of whose blocks are bad gets zeros. workspace as for duo_attn_decode
 * (duo_decode_workspace_size); o must not overlap q. */
duo_status duo_attn_decode_paged_varlen(duo_handle* handle, const duo_kv_cache* cache, const duo_paged* paged,
                                        const int32_t* seq_lens, int64_t max_len, const void* q, void* o,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* Dual Chunk Attention (vLLM pull request "[Model] Implement DualChunkAttention for
 * Qwen2 Models"): the sequence is cut into chunks of chunk_len positions from the start
 * (the last one may be shorter) and every position carries three query vectors made by
 * the rotary layer. Query i attends causally to every key j <= i with
 *     weight = (q_x(i) . k_j) * softmax_scale * mscale[i],   softmax_scale = 1/sqrt(D),
 * where q_x is q when j lies in i's chunk, q_succ when j lies in the chunk just before,
 * and q_inter for any earlier chunk; mscale is an fp32 per-position factor applied to
 * the fp32 product (NULL: 1). The pull request asks for this as one fused kernel in
 * place of three attention calls per chunk merged by log-sum-exp.
 *
 * Both entry points treat every head as full attention: the handle must have no
 * streaming head (DUO_ERR_UNSUPPORTED otherwise). chunk_len must be a positive multiple
 * of 256 (DUO_ERR_UNSUPPORTED otherwise) so that chunk boundaries fall on the
 * kernels' 256-row query blocks and 128-key tiles.
 *
 * duo_dca_prefill: prefill of T tokens at positions n ... n+T-1 against the cache as it
 * is before them (cache NULL or cache->n = 0: one-shot; else a chunk of a chunked
 * prefill, cache->n a multiple of 256, keys of rows [0, n) read from cache->k_full /
 * v_full). q, q_succ, q_inter: bf16 [B, T, Hq, D]; k, v: bf16 [B, T, Hkv, D]; mscale:
 * fp32 [B, T] (the chunk's positions) device memory or NULL; o: bf16 [B, T, Hq, D];
 * all device, 16-byte aligned. Append k and v with duo_kv_append afterwards. */
duo_status duo_dca_prefill(duo_handle* handle, const duo_kv_cache* cache, const void* q, const void* q_succ,
                           const void* q_inter, const void* k, const void* v, const float* mscale, int32_t T,
                           int32_t chunk_len, void* o, void* stream);

/* duo_dca_decode: one decode step at position cache->n - 1 (the token appended first)
 * over the retrieval caches. q, q_succ, q_inter: bf16 [B, Hq, D]; mscale: fp32 [B] or
 * NULL; o: bf16 [B, Hq, D]; workspace as for duo_attn_decode. */
duo_status duo_dca_decode(duo_handle* handle, const duo_kv_cache* cache, const void* q, const void* q_succ,
                          const void* q_inter, const float* mscale, int32_t chunk_len, void* o, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Per-sequence lengths on the device: serving batches
 * hold sequences of different lengths, and a decode step whose lengths live in device
 * memory can be captured once in a CUDA graph and replayed step after step. The
 * transformers pull request "[WIP] Dynamic length in static cache" debates exactly
 * this: a length the compiled step reads at run time instead of a host integer.
 *
 * duo_kv_append_varlen: appends ONE token to every sequence b at position
 * seq_lens[b] (int32 [B], device memory, read and then advanced by one on the device).
 * k_new, v_new: bf16 [B, 1, Hkv, D]. Same slot rule as duo_kv_append. A sequence whose
 * retrieval cache is full is left unchanged and duo_device_error() reports
 * DUO_ERR_CAPACITY. cache->n is not used or changed. */
duo_status duo_kv_append_varlen(duo_handle* handle, duo_kv_cache* cache, int32_t* seq_lens, const void* k_new,
                                const void* v_new, void* stream);

/* duo_attn_decode with per-sequence lengths: sequence b holds seq_lens[b] tokens
 * (device int32 [B], values clamped to [0, max_len]) and its query is at position
 * seq_lens[b] - 1. The work split is planned for max_len (host, 1 ... max_seq_len),
 * so the launch shape does not depend on the device values; a sequence of length 0
 * gets a zero output. cache->n is not used. Workspace as for duo_attn_decode. */
duo_status duo_attn_decode_varlen(duo_handle* handle, const duo_kv_cache* cache, const int32_t* seq_lens,
                                  int64_t max_len, const void* q, void* o, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Synchronises the device, then returns (and clears) the OR of the error codes that
 * kernels of this library recorded when a bounded wait ran out, or when a device-side
 * append met a full cache; 0 = none. Sets *code and returns DUO_ERR_DEVICE_TIMEOUT if
 * a wait ran out, DUO_ERR_CAPACITY if the only error is a full cache. */
duo_status duo_device_error(uint32_t* code);

/* Self-test of failure detection (the pages have no counterpart): launches one
 * CTA that waits on an mbarrier nothing completes, with the same bounded wait
 * the attention kernels use but a limit of limit_us microseconds (1 ... 10^6).
 * The wait gives up and records an error code (1 << 16); a following duo_device_error()
 * returns DUO_ERR_DEVICE_TIMEOUT, and the CUDA context stays usable. A warp of the CTA then
 * waits together, its lanes' times ending apart; 1 << 17 is recorded as well if the lanes
 * come out with different answers. */
duo_status duo_selftest_bounded_wait(uint32_t limit_us, void* stream);

/* Message describing the last error of the calling host thread ("" if none). */
const char* duo_last_error(void);

/* Short name of a status code. */
const char* duo_status_string(duo_status status);

#ifdef __cplusplus
}
#endif

#endif /* DUO_ATTN_H_ */
