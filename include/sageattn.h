/*
 * sageattn.h — C ABI of libsageattn.so: SageAttention-style quantized attention forward,
 * O = softmax(Q K^T · sm_scale) V, for one NVIDIA GB300 (sm_103a).
 *
 * The operation (pwwt.cn "SageAttention deployment pitfalls guide"):
 *   §1   Q and K are quantized to INT8 with fine-grained scales and QK^T runs on the
 *        8-bit values; V is quantized to FP8 and P·V runs with FP16/FP32 accumulators;
 *        the output stays FP16/BF16.
 *   §4.1 sageattn(q, k, v, tensor_layout="HND"|"NHD", is_causal, sm_scale=None,
 *        return_lse): inputs FP16 or BF16 on one device with one dtype, last dimension
 *        contiguous; head_dim below 64 is zero-padded to 64, between 64 and 128 to 128,
 *        above 128 is an error; Hq must be a multiple of Hkv (GQA); Nq may differ from Nk.
 *   §4.2 qk_quant_gran (per_warp / per_thread; per_block added), pv_accum_dtype
 *        (fp16 / fp32 / fp16+fp32), smooth_k (subtract K's mean over the sequence),
 *        smooth_v (same for V).
 *   §4 (end) sageattn_varlen: variable-length batches given by cu_seqlens_q / cu_seqlens_k.
 *
 * Conventions for every entry point:
 *   - Pointers named "device" are CUDA device pointers on the current device; the caller
 *     owns every buffer (inputs, outputs, LSE, workspace). The library never allocates or
 *     frees device memory, never synchronises inside sage_attn / sage_attn_varlen, and
 *     enqueues all work on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   - Arguments are validated on the host before anything is launched: on a non-zero
 *     return nothing was written. Errors found on the device (a bad cu_seqlens, a value
 *     too large for the exact mean, a pipeline wait that timed out) are recorded in the
 *     workspace and read back with sage_read_device_status().
 *   - Strides are in elements. The channel (head_dim) stride is always 1.
 *   - The workspace must be 256-byte aligned, at least sage_attn_workspace_size() bytes,
 *     and must not be shared by calls that may run concurrently.
 *   - Thread safety: calls from several host threads are safe; the only global state is a
 *     per-device cache of the kernels' shared-memory opt-in (and of whether the device is
 *     supported). A cudaDeviceReset clears the opt-in but not the cache: do not reset a
 *     device the library has already launched on.
 */
#ifndef SAGEATTN_H
#define SAGEATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SAGE_OK = 0,
  SAGE_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad enum, Nk == 0 with Nq > 0 */
  SAGE_ERR_HEAD_DIM = 2,     /* head_dim < 1 or > 128 */
  SAGE_ERR_DTYPE = 3,        /* dtype not SAGE_F16 / SAGE_BF16 */
  SAGE_ERR_STRIDE = 4,       /* misaligned pointer or a stride that breaks the layout rules */
  SAGE_ERR_GQA = 5,          /* Hq not a multiple of Hkv */
  SAGE_ERR_WORKSPACE = 6,    /* workspace null, misaligned or too small */
  SAGE_ERR_RANGE = 7,        /* (device) |x| >= 2^38 / N: too large for the exact mean */
  SAGE_ERR_UNSUPPORTED = 8,  /* pv_accum_dtype SAGE_ACC_FP16 */
  SAGE_ERR_TIMEOUT = 9,      /* (device) a bounded pipeline wait expired */
  SAGE_ERR_CUDA = 10,        /* a CUDA runtime/driver call failed */
  SAGE_ERR_DEVICE = 11,      /* current device is not compute capability 10.3 */
  SAGE_ERR_SEQLENS = 12,     /* (device) cu_seqlens not non-decreasing / out of range */
  SAGE_ERR_PAGE = 13         /* (device) a page table entry outside of the cache */
} sage_status;

enum { SAGE_HND = 0, SAGE_NHD = 1 };                       /* §4.1 tensor_layout */
enum { SAGE_F16 = 0, SAGE_BF16 = 1 };                      /* input/output dtype */
enum { SAGE_F32 = 2 };                                     /* weights of sage_qk_norm_rope besides */
enum { SAGE_S8 = 0, SAGE_E4M3 = 1 };                       /* codes of an 8-bit cache */
enum { SAGE_PER_BLOCK = 0, SAGE_PER_WARP = 1, SAGE_PER_THREAD = 2 };   /* qk_quant_gran */
enum { SAGE_ACC_FP32 = 0, SAGE_ACC_FP16_FP32 = 1, SAGE_ACC_FP32_FP32 = 2, SAGE_ACC_FP16 = 3 };

/* A 4-d FP16/BF16 device tensor in the order the call's tensor_layout names:
 * HND = [batch, heads, seq, head_dim], NHD = [batch, seq, heads, head_dim].
 * stride[0..2] are the element strides of the first three dimensions; the fourth
 * (channel) stride is 1. `data` points at element [0, 0, 0, 0]. */
typedef struct {
  void* data;
  int64_t stride[3];
} sage_tensor;

/* A packed variable-length FP16/BF16 device tensor [total_tokens, heads, head_dim]
 * with element strides per token and per head; the channel stride is 1. */
typedef struct {
  void* data;
  int64_t stride_token;
  int64_t stride_head;
} sage_packed;

/* Bytes of workspace sage_attn needs for these sizes (0 on invalid sizes). */
size_t sage_attn_workspace_size(int batch, int heads_q, int heads_kv, int seqlen_q,
                                int seqlen_k, int head_dim, int qk_quant_gran);

/* Dense forward (§4.1, §4.2).
 *   q [B, Hq, Nq, d] / [B, Nq, Hq, d]; k, v [B, Hkv, Nk, d] / [B, Nk, Hkv, d] (device,
 *   read only); out: same shape and layout as q (device, written, dtype = input dtype).
 *   lse: device float [B, Hq, Nq] contiguous, natural-log log-sum-exp of the scaled
 *   scores sm_scale·q·k over the allowed keys; written only when return_lse != 0
 *   (may be NULL otherwise).
 *   is_causal: key j is allowed for query i iff j <= i (top-left aligned, as
 *   torch.nn.functional.scaled_dot_product_attention).
 *   sm_scale: scale of the scores; NaN or <= 0 selects 1/sqrt(head_dim).
 *   qk_quant_gran: token groups sharing one INT8 scale — per_block 128 Q rows / 64 K rows,
 *   per_warp 32 / 64, per_thread 1 / 16.
 *   pv_accum_dtype: SAGE_ACC_FP32, SAGE_ACC_FP32_FP32 or SAGE_ACC_FP16_FP32, one
 *   arithmetic on this GPU: P is scaled by 448 before its FP8 rounding and P·V accumulates
 *   in fp32 over every key (§4.2 ranks fp16 accumulation fastest and fp32 most stable, with
 *   fp16+fp32 between them; the tensor cores here accumulate fp16 no faster than fp32, so the
 *   compromise is taken at fp32); SAGE_ACC_FP16 returns SAGE_ERR_UNSUPPORTED.
 *   smooth_k / smooth_v: subtract the per-(batch, head, channel) mean over the sequence.
 *   Nq == 0 or B == 0 is a no-op returning SAGE_OK.
 * Returns a sage_status. */
int sage_attn(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
              const sage_tensor* out, float* lse, int batch, int heads_q, int heads_kv,
              int seqlen_q, int seqlen_k, int head_dim, int dtype, int tensor_layout,
              int is_causal, float sm_scale, int return_lse, int qk_quant_gran,
              int pv_accum_dtype, int smooth_k, int smooth_v, void* workspace,
              size_t workspace_bytes, void* stream);

/* FP16 P·V variant (pwwt.cn "SageAttention deployment pitfalls guide" §5.3–§5.4: the INT8-QK
 * + FP16-PV kernel, the quality fallback with FP8 turned off): as sage_attn, with the same
 * arguments, workspace size and errors, except that V' = V - v̄ is kept in fp16 (no per-channel
 * scale) and P = 2^(t - m) is rounded to fp16 (σ_P = 1); both P·V operands are fp16 on the
 * tensor cores (kind::f16) with fp32 accumulation. pv_accum_dtype: SAGE_ACC_FP32,
 * SAGE_ACC_FP32_FP32 or SAGE_ACC_FP16_FP32 (one arithmetic, as for sage_attn);
 * SAGE_ACC_FP16 returns SAGE_ERR_UNSUPPORTED. |V - v̄| beyond the fp16 range becomes ±inf. */
int sage_attn_qk_int8_pv_fp16(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
                              const sage_tensor* out, float* lse, int batch, int heads_q,
                              int heads_kv, int seqlen_q, int seqlen_k, int head_dim, int dtype,
                              int tensor_layout, int is_causal, float sm_scale, int return_lse,
                              int qk_quant_gran, int pv_accum_dtype, int smooth_k, int smooth_v,
                              void* workspace, size_t workspace_bytes, void* stream);

/* FP4 microscaled variant (pwwt.cn "SageAttention deployment pitfalls guide" §5.5: the
 * SageAttention3 kernel for Blackwell, "FP4 microscaling"; the guide names only its API,
 * sageattn3_blackwell(q, k, v, is_causal)): as sage_attn, with the same arguments, workspace
 * size and errors, except for the quantisation:
 *   Q and K' = K - k̄: each token group (qk_quant_gran) is mapped onto [-448, 448] by its
 *   scale g = absmax / 448; every 16 channels of a row share an E4M3 block scale s (the
 *   block's largest mapped magnitude, rounded) and each element is the E2M1 code of
 *   fl32(u · fl32(6 / s)), RNE, saturating at ±6.
 *   V' = V - v̄: each channel is mapped by absmax_c / 448 and blocked over 16 tokens.
 *   P: 448 · 2^(t - m), blocked over 16 keys.
 * Every E2M1 code times its E4M3 block scale is exact in fp16, so both products run on
 * fp16 tensor cores (kind::f16) and give what a block-scaled FP4 product gives. P·V
 * accumulates in fp32; pv_accum_dtype as for sage_attn. Dense problems only. */
int sage_attn_fp4(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
                  const sage_tensor* out, float* lse, int batch, int heads_q, int heads_kv,
                  int seqlen_q, int seqlen_k, int head_dim, int dtype, int tensor_layout,
                  int is_causal, float sm_scale, int return_lse, int qk_quant_gran,
                  int pv_accum_dtype, int smooth_k, int smooth_v, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Capacity of the scratch array built into the library for sage_attn_no_alloc. */
#define SAGE_NO_ALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/* sage_attn without a caller-supplied workspace and without any device allocation.
 * (The pages have no counterpart; this exists for callers that cannot allocate.)
 * Some callers cannot call cudaMalloc where they run attention: a plugin executing inside a
 * host engine that gives it only its input/output buffers and forbids allocation while it
 * runs, or a latency-critical path that cannot afford an allocation's time or failure. This
 * entry point takes its scratch from a fixed array of SAGE_NO_ALLOC_SCRATCH_BYTES bytes
 * compiled into the library (held by every GPU that loads the library until the process
 * exits); the caller still passes inputs, outputs and the optional LSE buffer.
 *   Arguments, layouts and results are those of sage_attn.
 *   Returns SAGE_ERR_WORKSPACE, before launching anything, when the problem needs more than
 *   SAGE_NO_ALLOC_SCRATCH_BYTES of scratch (sage_attn_workspace_size tells how much).
 *   Arguments are checked first, with sage_attn's rules and error codes.
 *   The first call on each device looks up the array's device address (cudaGetSymbolAddress,
 *   with that device current) and caches it for the life of the process; make that first
 *   call before any stream capture. After a cudaDeviceReset the cached address is stale:
 *   do not call this entry point in a process that has reset a device it used.
 *   Every call on a device uses the same array: calls that may overlap on the GPU (other
 *   streams, other host threads) race and must be serialised by the caller. Each call
 *   clears what it needs cleared; nothing an earlier call left in the array is read.
 *   Calls no cudaMalloc, cudaFree or allocating library routine. */
int sage_attn_no_alloc(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
                       const sage_tensor* out, float* lse, int batch, int heads_q, int heads_kv,
                       int seqlen_q, int seqlen_k, int head_dim, int dtype, int tensor_layout,
                       int is_causal, float sm_scale, int return_lse, int qk_quant_gran,
                       int pv_accum_dtype, int smooth_k, int smooth_v, void* stream);

/* Bytes of workspace sage_attn_varlen needs (0 on invalid sizes). */
size_t sage_attn_varlen_workspace_size(int batch, int heads_q, int heads_kv, int total_q,
                                       int total_k, int head_dim, int qk_quant_gran);

/* Variable-length forward (§4, sageattn_varlen). Sequence b owns query tokens
 * [cu_seqlens_q[b], cu_seqlens_q[b+1]) of q and key tokens [cu_seqlens_k[b],
 * cu_seqlens_k[b+1]) of k and v; smoothing means, quantisation groups and the causal mask
 * restart per sequence.
 *   q, out: [total_q, Hq, d]; k, v: [total_k, Hkv, d] (device).
 *   cu_seqlens_q, cu_seqlens_k: device int32 [batch + 1], non-decreasing, starting at 0
 *   and ending at total_q / total_k (checked on the device: SAGE_ERR_SEQLENS).
 *   max_seqlen_q / max_seqlen_k: upper bounds of the lengths (checked on the device).
 *   lse: device float [Hq, total_q] when return_lse != 0.
 *   A sequence with no keys but some queries is a device error (SAGE_ERR_SEQLENS).
 * Other arguments as sage_attn. */
int sage_attn_varlen(const sage_packed* q, const sage_packed* k, const sage_packed* v,
                     const sage_packed* out, float* lse, const int32_t* cu_seqlens_q,
                     const int32_t* cu_seqlens_k, int batch, int max_seqlen_q,
                     int max_seqlen_k, int total_q, int total_k, int heads_q, int heads_kv,
                     int head_dim, int dtype, int is_causal, float sm_scale, int return_lse,
                     int qk_quant_gran, int pv_accum_dtype, int smooth_k, int smooth_v,
                     void* workspace, size_t workspace_bytes, void* stream);

/* The FP16 P·V variant of sage_attn_varlen (see sage_attn_qk_int8_pv_fp16): same arguments,
 * workspace size and errors; V' and P in fp16 on the tensor cores. */
int sage_attn_varlen_qk_int8_pv_fp16(const sage_packed* q, const sage_packed* k,
                                     const sage_packed* v, const sage_packed* out, float* lse,
                                     const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                     int batch, int max_seqlen_q, int max_seqlen_k, int total_q,
                                     int total_k, int heads_q, int heads_kv, int head_dim,
                                     int dtype, int is_causal, float sm_scale, int return_lse,
                                     int qk_quant_gran, int pv_accum_dtype, int smooth_k,
                                     int smooth_v, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Composition of partial results over disjoint key sets (pwwt.cn "SageAttention deployment
 * pitfalls guide" §4.1: return_lse exists for Ring Attention and similar schemes, which attend
 * to chunks of the keys separately). For every (b, h, n) row:
 *   lse = ln sum_i exp(lse_i),   out = sum_i exp(lse_i - lse) * out_i
 * computed in fp32 and rounded once to `dtype`.
 *   outs[0..n_parts): device tensors in `tensor_layout` (as sage_attn's out, dtype `dtype`);
 *   lses[0..n_parts): device float [B, H, N] contiguous (as sage_attn writes them);
 *   out: device tensor of the same shape (may alias outs[0]); lse_out: device float
 *   [B, H, N] or NULL. The pointer arrays themselves are host memory.
 * A part whose lse is -inf contributes nothing; a row no part sees gets out = 0 and
 * lse = -inf. 1 <= n_parts <= SAGE_MAX_MERGE_PARTS. Errors: SAGE_ERR_INVALID_ARG (counts,
 * null pointers, layout), SAGE_ERR_DTYPE, SAGE_ERR_HEAD_DIM, SAGE_ERR_STRIDE (pointer not
 * 2-byte aligned, negative stride), SAGE_ERR_CUDA. Nothing is launched for an empty problem. */
#define SAGE_MAX_MERGE_PARTS 16
int sage_merge_partials(const sage_tensor* outs, const float* const* lses, int n_parts,
                        const sage_tensor* out, float* lse_out, int batch, int heads,
                        int seqlen, int head_dim, int dtype, int tensor_layout, void* stream);

/* ---- Attention with modified scores, on 16-bit operands ----
 * For the layers that the quantised calls cannot take: capped or biased scores, document and
 * prefix masks.
 *   s_ij = sm_scale q_i.k_j;  softcap > 0: s = softcap tanh(s / softcap);
 *   slopes: s -= slopes[h] |i + q_offset - j|
 *   visible(i, j) = (!is_causal || j <= i + q_offset || j < prefix_lens[b])
 *                   && (no documents || (doc_q[b][i] == doc_k[b][j] && doc_k[b][j] >= 0))
 *   out_i = sum_j softmax over the visible j of s_ij, times v_j;  lse_i = ln sum_j exp s_ij
 * Q K^T and P V are products of the inputs' type with fp32 sums; the softmax is fp32, and its weights
 * are rounded once to the inputs' type for P V. A row that sees no key gets out = 0 and lse = -inf, and
 * so does a row all of whose visible scores are -inf.
 *   q, k, v, out, tensor_layout, is_causal, sm_scale, lse, return_lse: as sage_attn. q_offset shifts the
 *   queries' positions (the next chunk of a prompt: the number of keys before it); it may be negative. No position and,
 *   with slopes, no distance may pass 2^31 - 256: -2^31 + 256 <= q_offset (with slopes: q_offset - Nk) and
 *   q_offset + Nq <= 2^31 - 256, or SAGE_ERR_INVALID_ARG.
 *   softcap: 0 (none) or up to 4096. slopes: device float [Hq] or NULL. prefix_lens: device int32 [B] or NULL; only with is_causal.
 *   doc_q [B, Nq], doc_k [B, Nk]: device int32, contiguous, both or neither. A negative id is padding,
 *   which sees nothing and is seen by nothing. Rows of k and v that are padding, or that lie behind the
 *   last key any row sees under the causal and prefix masks (a buffer longer than what it
 *   holds), may hold anything; every other row of v must be finite (a weight of 0 times an infinity is NaN
 *   in the rows that do not see it).
 *   workspace: sage_scored_attn_workspace_size() bytes; `packed` != 0 where q, k and v all have 16-byte
 *   aligned rows (address, and strides and head_dim multiples of 8 elements; no zero stride of a
 *   dimension longer than 1) and need no padded copy there; `packed` + 2 where there are no documents. Where no more
 *   than SAGE_STATUS_BYTES are needed, workspace may be NULL: no status is kept then.
 * Nq == 0 or B == 0 is a no-op; Nk == 0 writes 0 and -inf. */
size_t sage_scored_attn_workspace_size(int batch, int heads_q, int heads_kv, int seqlen_q, int seqlen_k,
                                       int head_dim, int packed);
int sage_scored_attn(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
                     const sage_tensor* out, float* lse, const float* slopes,
                     const int32_t* prefix_lens, const int32_t* doc_q, const int32_t* doc_k, int batch,
                     int heads_q, int heads_kv, int seqlen_q, int seqlen_k, int head_dim, int dtype,
                     int tensor_layout, int is_causal, float sm_scale, float softcap, int q_offset,
                     int return_lse, void* workspace, size_t workspace_bytes, void* stream);

/* ---- A paged key-value cache ----
 * k, v: device FP16/BF16 [num_pages, Hkv, page_size, d] (HND) or [num_pages, page_size, Hkv, d] (NHD), any
 * strides of the first three dimensions (k_stride, v_stride, in that order), channel stride 1.
 * Token slot t of sequence b lies in page page_table[b * table_stride + t / page_size] at
 * t % page_size; page_table has max_pages entries per row (at most 2^31 - 65536 slots), of which only those
 * of held tokens are read. seq_lens: device int32 [batch], the tokens each sequence holds.
 * mass: device float [num_pages, Hkv, page_size] contiguous, the attention weight each token has drawn,
 * or NULL. positions: device int32 of the same shape, the tokens' positions, or NULL (the slot).
 * Errors found on the device: SAGE_ERR_SEQLENS (a length outside of [0, max_seqlen] or of the table's
 * room: the sequence counts as empty), SAGE_ERR_PAGE (an entry outside of [0, num_pages): its tokens
 * count as zero rows, are not written and not moved). Nothing outside of the cache is touched. */
typedef struct {
  void* k;
  int64_t k_stride[3];
  void* v;
  int64_t v_stride[3];
  int num_pages, page_size;
  const int32_t* page_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* seq_lens;
  float* mass;
  int32_t* positions;
} sage_paged_cache;

#define SAGE_STATUS_BYTES ((size_t)256) /* workspace of a call that needs only its status word */

/* Attention of one new token per sequence over its held tokens (its own K and V appended before).
 * Scores as sage_scored_attn's: capped, then biased by slopes[h] |q_position - position of the key|.
 *   q, out: [batch, Hq, d] (stride_token is the sequence's); lse: device float [batch, Hq] or NULL.
 *   slopes: device float [Hq] or NULL; q_positions: device int32 [batch] or NULL (seq_len - 1).
 *   max_seqlen: an upper bound of seq_lens. cache->mass, where not NULL: each held token's weight,
 *   summed over the query heads of its key/value head, is added. A page that several
 *   sequences share is given the weights of all, in no fixed order. workspace: as sage_scored_attn's;
 *   with mass it holds 4 batch Hq max_seqlen bytes of scores.
 *   Once a sequence has been evicted from, its slots and its length are no positions: slopes then need
 *   cache->positions and q_positions.
 * A sequence that holds nothing gets out = 0 and lse = -inf. */
size_t sage_paged_attn_workspace_size(int batch, int heads_q, int heads_kv, int max_seqlen,
                                      int head_dim, int accumulate);
int sage_paged_attn(const sage_packed* q, const sage_paged_cache* cache, const sage_packed* out,
                    float* lse, const float* slopes, const int32_t* q_positions, int batch,
                    int heads_q, int heads_kv, int max_seqlen, int head_dim, int dtype,
                    int tensor_layout, float sm_scale, float softcap, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Writes new tokens behind the held ones: token t of k, v [tokens, Hkv, d] belongs to the sequence b with
 * cu_seqlens[b] <= t < cu_seqlens[b + 1] and goes to slot seq_lens[b] + t - cu_seqlens[b]. seq_lens is
 * read, not raised. cu_seqlens: device int32 [batch + 1], non-decreasing from 0; NULL: one token per
 * sequence (tokens == batch). Tokens from cu_seqlens[batch] on are left out, and so are all tokens of a
 * sequence of negative length, and those whose slot lies behind the table's room or whose page is not in the
 * cache (SAGE_ERR_SEQLENS, SAGE_ERR_PAGE). cache->mass becomes 0 in the written slots
 * and cache->positions the token's entry of `positions` (device int32 [tokens]) or its slot, which is no
 * position once the sequence has been evicted from (it lies below the kept ones). Two
 * tokens must not share a slot. workspace: NULL, or SAGE_STATUS_BYTES for the device status. */
int sage_paged_append(const sage_packed* k, const sage_packed* v, const sage_paged_cache* cache,
                      const int32_t* cu_seqlens, const int32_t* positions, int batch, int tokens,
                      int heads_kv, int head_dim, int dtype, int tensor_layout, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Cuts every sequence that holds more than `budget` tokens down to `budget`, for each key/value head by
 * itself: tokens with a position below `sink` or within the last `recent` of the head's largest
 * position stay, then those with the largest mass (ties: the lowest slot; NaN counts as -inf). Kept
 * tokens from slot `budget` on move, in order, into the freed slots below it, with their mass and
 * position; slots from `budget` on keep what they held. new_lens: device int32 [batch], written
 * min(seq_len, budget), or seq_len where an error is found: that sequence is left as it was; it must not
 * overlap seq_lens. cache->mass and cache->positions are needed where there are pages. Each page belongs to one sequence.
 * Only sage_paged_attn adds mass: right after a prompt the lowest of the unprotected slots stay.
 * budget >= 1, sink + recent <= budget (where positions repeat and more than `budget` tokens would
 * have to stay, those of the lowest slots do). */
size_t sage_paged_evict_workspace_size(int batch, int heads_kv, int max_seqlen, int budget);
int sage_paged_evict(const sage_paged_cache* cache, int32_t* new_lens, int batch, int heads_kv,
                     int max_seqlen, int head_dim, int dtype, int tensor_layout, int budget, int sink,
                     int recent, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Serving from an 8-bit cache: norms and rotation, page tables, append, read, attention ---- */

/* Norms of queries and keys for each (token, head) row and their rotation by position, in one pass:
 *   y = x / sqrt(mean(x^2) + eps) * w;  pairs p < rot_dim / 2 of channels (p, p + rot_dim / 2), or
 *   (2 p, 2 p + 1) with interleaved, turned by position * inv_freq[p]:
 *   (y_i cos a - y_j sin a, y_j cos a + y_i sin a). Channels from rot_dim on are not turned.
 *   q, q_out: Hq heads of `seqlen` tokens as sage_attn's q; k, k_out: Hkv heads of the same tokens. An
 *   output may be its input (the same address and strides), and must not overlap an input otherwise.
 *   positions: device int32, token i of batch b at b positions_stride + i; NULL: i. inv_freq: device
 *   float [rot_dim / 2] (NULL with rot_dim 0). q_weight, k_weight: device [head_dim] of `dtype` or SAGE_F32
 *   (weight_dtype), or NULL for ones. Squares are summed in fp32: magnitudes below 1e18; with eps below
 *   2^-90, where small rows matter, any.
 * Angles are taken as 64-bit fractions of a turn, off by at most 2^-52 of themselves and 2^-65 of a turn for
 * each step of the position.
 * batch * seqlen below 2^31; rot_dim even, 0 to head_dim. */
int sage_qk_norm_rope(const sage_tensor* q, const sage_tensor* k, const sage_tensor* q_out,
                      const sage_tensor* k_out, const int32_t* positions, int64_t positions_stride,
                      const float* inv_freq, const void* q_weight, const void* k_weight,
                      int weight_dtype, int batch, int heads_q, int heads_kv, int seqlen, int head_dim,
                      int rot_dim, int dtype, int tensor_layout, int interleaved, float eps,
                      void* stream);

/* Pages for sequences that grow, from a stack of free ones: the first *free_count entries of
 * free_pages [num_pages] (device int32). Sequence b holds seq_lens[b] tokens and is to hold add_lens[b]
 * more (device int32 [batch]). In the order of the sequences, each takes the pages it lacks from the top of the
 * stack into its row of page_table; once one finds too few, it and all later ones that need pages take
 * none. Table entries of pages that are held already, or behind the last, are not touched.
 *   new_lens [batch]: seq_lens + add_lens where served, seq_lens otherwise; held_lens [batch]: seq_lens
 *   where served, -1 otherwise (the appends leave such tokens out); cu_seqlens [batch + 1]: where the new tokens
 *   of each sequence lie in packed rows, served or not; positions [max_tokens]: next_positions[b] (NULL:
 *   seq_lens[b]) + the token's place, -1 behind the last; slots [max_tokens] (int64): page * page_size +
 *   place in the page of each new token, -1 where it has none; new_free_count [1]. All device, none of
 *   them an input.
 * A sequence whose lengths are negative, exceed its row of the table, or whose new tokens end behind
 * max_tokens is not served (SAGE_ERR_SEQLENS, as for a count outside of [0, num_pages], which is clamped;
 * a held page outside of the cache leaves its slot -1: SAGE_ERR_PAGE). workspace: NULL or
 * SAGE_STATUS_BYTES. */
int sage_paged_assign(int32_t* page_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                      const int32_t* add_lens, const int32_t* next_positions, const int32_t* free_pages,
                      const int32_t* free_count, int num_pages, int page_size, int batch, int max_tokens,
                      int32_t* new_lens, int32_t* held_lens, int32_t* cu_seqlens, int32_t* positions,
                      int64_t* slots, int32_t* new_free_count, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Pages of sequences that shrink, back onto the stack: of the seq_lens[b] tokens that sequence b holds
 * keep_lens[b] stay; the pages behind them are written to free_pages from *free_count on, in the order of
 * the sequences and of their rows. The table is not changed. A page belongs to one sequence: one that two
 * hold would come back twice. A sequence with lengths out of range or
 * keep_lens > seq_lens (SAGE_ERR_SEQLENS), or with a page among those given that is not in
 * [0, num_pages) (SAGE_ERR_PAGE), gives none; where the stack has no room, that sequence and the later ones
 * do not either (SAGE_ERR_SEQLENS). */
size_t sage_paged_release_workspace_size(int batch);
int sage_paged_release(const int32_t* page_table, int64_t table_stride, int max_pages,
                       const int32_t* seq_lens, const int32_t* keep_lens, int32_t* free_pages,
                       const int32_t* free_count, int num_pages, int page_size, int batch,
                       int32_t* new_free_count, void* workspace, size_t workspace_bytes, void* stream);

/* A paged cache in 8 bits. As sage_paged_cache, with codes of k_type / v_type (SAGE_S8, SAGE_E4M3; strides in
 * elements) and k_scales / v_scales: device float [num_pages, Hkv, page_size / block], contiguous; `block`
 * divides page_size. Slot t of a page has the scale t / block; a value is code * scale. */
typedef struct {
  void* k;
  int64_t k_stride[3];
  void* v;
  int64_t v_stride[3];
  float* k_scales;
  float* v_scales;
  int k_type, v_type;
  int num_pages, page_size, block;
  const int32_t* page_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* seq_lens;
} sage_q8_cache;

/* Writes new tokens behind the held ones, as sage_paged_append, into an 8-bit cache. With x the block's new
 * tokens of a head and s the scale of the earlier ones (0 where the block starts with a new token), the
 * scale becomes max(s, need, 2^-100), need = max|x| / 127 for int8, the smallest power of two with
 * max|x| <= 448 need for E4M3; codes are x / scale rounded to nearest even (as x times fl32(1 / scale)), and
 * where the scale grew the earlier codes become code * fl32(s / scale), rounded again. k and v must be finite.
 * Two sequences must not append to one block. */
int sage_paged_append_q8(const sage_packed* k, const sage_packed* v, const sage_q8_cache* cache,
                         const int32_t* cu_seqlens, int batch, int tokens, int heads_kv, int head_dim,
                         int dtype, int tensor_layout, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Values of held tokens in 16 bits: row t of k_out, v_out [tokens, Hkv, d] with cu_seqlens[b] <= t <
 * cu_seqlens[b + 1] is slot starts[b] + t - cu_seqlens[b] of sequence b (starts: device int32 [batch] or
 * NULL for 0). Rows of no held token (behind seq_lens, SAGE_ERR_SEQLENS; of a page outside of the cache,
 * SAGE_ERR_PAGE; behind the last sequence) become 0. workspace: NULL or SAGE_STATUS_BYTES. */
int sage_paged_read_q8(const sage_packed* k_out, const sage_packed* v_out, const sage_q8_cache* cache,
                       const int32_t* cu_seqlens, const int32_t* starts, int batch, int tokens,
                       int heads_kv, int head_dim, int dtype, int tensor_layout, void* workspace,
                       size_t workspace_bytes, void* stream);

/* sage_paged_attn over an 8-bit cache; positions of keys are their slots. Scales must be finite and not
 * negative. Weights are rounded to fp16 once, whatever q's type. */
size_t sage_paged_attn_q8_workspace_size(int batch, int heads_q, int heads_kv, int max_seqlen,
                                         int head_dim);
int sage_paged_attn_q8(const sage_packed* q, const sage_q8_cache* cache, const sage_packed* out, float* lse,
                       const float* slopes, const int32_t* q_positions, int batch, int heads_q,
                       int heads_kv, int max_seqlen, int head_dim, int dtype, int tensor_layout,
                       float sm_scale, float softcap, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Human-readable name of a sage_status. Never NULL. */
const char* sage_status_string(int status);

/* Name and description of the CUDA error behind the calling thread's most recent
 * SAGE_ERR_CUDA ("no error" if there was none). Never NULL. */
const char* sage_last_cuda_error(void);

/* Synchronises `stream`, then returns the status the device recorded in `workspace`
 * during the last call that used it (SAGE_OK if none), or SAGE_ERR_CUDA. */
int sage_read_device_status(const void* workspace, void* stream);

/* 1 if the current CUDA device is compute capability 10.3 (GB300), else 0. */
int sage_device_supported(void);

/* Stage timing (off by default). While enabled, every sage_attn / sage_attn_varlen call
 * records CUDA events on its stream around its three stages (statistics, quantisation,
 * attention kernel); up to 8192 calls are kept. sage_profile_read synchronises those events
 * and writes the summed milliseconds per stage to stage_ms[0..2] and the number of calls to
 * *calls; it also clears the record. Enabling allocates CUDA events (no device memory).
 * Returns a sage_status. */
int sage_profile_enable(int on);
int sage_profile_read(double* stage_ms, int* calls);

/* ---- Test exports. They run the same kernels as the entry points above. ---- */

/* Copies the quantised state that the last sage_attn call with these sizes left in
 * `workspace` into canonical host-layout device buffers (all device, caller-owned):
 *   q8 int8 [B, Hq, Nq, d], sq float [B, Hq, ceil(Nq / Gq)],
 *   k8 int8 [B, Hkv, Nk, d], sk float [B, Hkv, ceil(Nk / Gk)],
 *   kmean, vmean, vscale float [B, Hkv, d], v8 uint8 E4M3 [B, Hkv, Nk, d].
 * Any output pointer may be NULL to skip it. */
int sage_debug_export_quant(const void* workspace, int batch, int heads_q, int heads_kv,
                            int seqlen_q, int seqlen_k, int head_dim, int qk_quant_gran,
                            int8_t* q8, float* sq, int8_t* k8, float* sk, float* kmean,
                            float* vmean, float* vscale, uint8_t* v8, void* stream);

/* sage_attn that additionally writes the integer scores S = Q8 · K8^T, exactly as the
 * attention kernel reads them from tensor memory, to `scores` (device int32
 * [B, Hq, Nq, Nk]; entries the causal mask skips are left untouched). */
int sage_attn_debug_scores(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v,
                           const sage_tensor* out, float* lse, int batch, int heads_q,
                           int heads_kv, int seqlen_q, int seqlen_k, int head_dim, int dtype,
                           int tensor_layout, int is_causal, float sm_scale, int return_lse,
                           int qk_quant_gran, int pv_accum_dtype, int smooth_k, int smooth_v,
                           void* workspace, size_t workspace_bytes, int32_t* scores,
                           void* stream);

/* Test hook: while `on` is non-zero, the attention kernel's producer issues no K/V tile
 * loads, so the consumers' bounded waits expire (about 2 s) and the device status becomes
 * SAGE_ERR_TIMEOUT; the kernel still exits cleanly and the context stays usable. Process-wide;
 * not for concurrent use. Returns SAGE_OK. */
int sage_debug_stall_attention(int on);

/* Which implementation dense sage_attn calls use. The main pipeline is the statistics,
 * finalisation, quantisation and tcgen05 attention kernels (four launches); the short-sequence
 * kernel (pnsm.cn §10: below about 1K tokens fixed costs dominate) takes problems with at most
 * 256 keys and 1024 queries in one launch, doing the statistics, quantisation and attention per
 * CTA of 128 query rows with the same arithmetic and results within the same tolerances.
 *   0 (default): the short-sequence kernel for such problems at head_dim <= 64 on a stream that
 *      is not capturing a CUDA graph, the main pipeline otherwise (measured faster in each
 *      case: 28 us against 37 per direct call at 256 keys; 22 us against 27 replayed);
 *   1: always the main pipeline;
 *   2: the short-sequence kernel whenever the problem fits it.
 * The FP16 P·V and FP4 variants and calls with the score dump, trace or stall hooks always take
 * the main pipeline. Process-wide; not for concurrent use. Returns SAGE_OK, or
 * SAGE_ERR_INVALID_ARG for another value. */
int sage_debug_select_path(int path);

/* Pipeline trace hook: while `clocks` (device, 4*64*8 int64, caller-owned) is non-NULL, dense
 * calls record clock64() of the first CTA's pipeline events there: [role][tile][event] with
 * role 0/1 = softmax of query tile A/B (events: scores ready, scores loaded, max done,
 * exponentials done, P buffer free, P written, O rescaled; event 7 of the last tile: output
 * written), role 2 = MMA issue (per tile x:
 * 4x+0 P ready, 4x+1 QK^T issued, 4x+2 O ready, 4x+3 P.V issued), role 3 = TMA (K, V
 * issued), for the first 64 KV tiles. NULL turns it off. Process-wide. Returns SAGE_OK.
 * The events are recorded by a separate test build of the E4M3 P·V attention kernel (the
 * production build carries no trace points, so its timing differs); calls of the FP16 P·V
 * and FP4 variants record nothing. */
int sage_debug_trace_attention(long long* clocks);

/* Converts n floats (device) to FP8 E4M3 (device bytes) with the round-to-nearest-even,
 * saturating conversion the kernels use for V and P. */
int sage_debug_e4m3(const float* x, uint8_t* out, int64_t n, void* stream);

/* Converts n floats (device) to FP4 E2M1 codes (device bytes, low 4 bits) with the
 * round-to-nearest-even conversion saturating at ±6 that the FP4 variant uses. */
int sage_debug_e2m1(const float* x, uint8_t* out, int64_t n, void* stream);

/* Copies the fp16 operands the attention kernel consumed after a dense call of the FP16 P·V
 * or FP4 variant into canonical layouts (device buffers of fp16 bit patterns):
 *   q16 [B, Hq, Nq, d] and k16 [B, Hkv, Nk, d] (the FP4 carriers; INT8 codes as fp16 after
 *   the other dense calls), v16 [B, Hkv, Nk, d] (V' in fp16, or the FP4 carriers of V).
 * Any output pointer may be NULL to skip it. */
int sage_debug_export_fp16(const void* workspace, int batch, int heads_q, int heads_kv,
                           int seqlen_q, int seqlen_k, int head_dim, int qk_quant_gran,
                           uint16_t* q16, uint16_t* k16, uint16_t* v16, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAGEATTN_H */
