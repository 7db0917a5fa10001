/*
 * mha.h -- C ABI of the GB300 (sm_103a) multi-head attention forward library.
 *
 * The operation is the forward pass of the Transformer's multi-head attention
 * sublayer, as the pages define it:
 *
 *   "003-Transformer" tutorial, section "Multi-head attention",
 *   MultiHeadedAttention.forward(query, key, value, mask):
 *     Q = query W_q^T + b_q, K = key W_k^T + b_k, V = value W_v^T + b_v
 *         (nn.Linear(d_model, d_model), weights stored [out, in]);
 *     each viewed as (B, L, h, d_k) and transposed to (B, h, L, d_k), so head i
 *         owns features [i*d_k, (i+1)*d_k), with d_k = d_model / h;
 *     per head: "The Annotated Transformer", section "Attention", attention():
 *         scores = Q K^T / sqrt(d_k); scores.masked_fill(mask == 0, -1e9);
 *         p_attn = softmax(scores, dim=-1); head = p_attn V;
 *     heads transposed back and concatenated to (B, L_q, h*d_k);
 *     out = concat W_o^T + b_o.
 *
 * Mask (1 = may attend): the AND of up to three parts, broadcast over heads
 * (mask.unsqueeze(1) in MultiHeadedAttention.forward):
 *   causal          key j allowed for query i iff j <= i ("The Annotated
 *                   Transformer", subsequent_mask(); diagonal allowed).
 *   key_valid_lens  key j allowed iff j < key_valid_lens[b] (d2l
 *                   MultiHeadAttention valid_lens, d2l Transformer chapter).
 *   dense           byte mask [B, dense_mq, L_k], dense_mq in {1, L_q};
 *                   0 = masked; dense_mq == 1 broadcasts over queries.
 * A masked score is REPLACED by -1e9 after the 1/sqrt(d_k) scaling, so a
 * query row whose keys are all masked gets uniform weights 1/L_k over all L_k
 * keys. Dropout is the identity (forward / evaluation).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers into buffers the caller owns,
 *     row-major and contiguous, unless an entry point says otherwise. The
 *     library never allocates or frees device memory and never synchronises
 *     the stream (except mha_check_device_status, which says so).
 *   - dt selects the storage type of query/key/value/weights/biases/out and of
 *     the workspace tensors: MHA_F32 (fp32 everywhere, fp32 SIMT arithmetic,
 *     any d_k <= 256) or MHA_BF16 (bf16 storage, fp32 accumulation on the
 *     tensor cores, d_k = 64 or 128, or d_k = 8, 16, 32 when d_model is a
 *     multiple of 64 (those heads run on the d_k = 64 kernels, zero-padded to 64
 *     columns on load); mha_forward and mha_forward_noalloc also take any other
 *     d_k <= 256 in bf16, which they run on the fp32 kernels over fp32 copies held
 *     in the workspace, then round the output to bf16).
 *     p_attn is always fp32.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the call returns without waiting for it.
 *   - Arguments are validated on the host before anything is enqueued. On a
 *     non-OK status returned by validation, no output buffer is touched.
 *     mha_last_error() then gives a message (thread-local).
 *   - B, L_q, L_k, d_model, h >= 1; d_model % h == 0 (the pages assert
 *     embedding_dim % head == 0). causal requires L_q == L_k (the subsequent
 *     mask is square).
 *   - MHA_BF16 also requires every tensor pointer to be 16-byte aligned.
 */
#ifndef GB300_MHA_H
#define GB300_MHA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MHA_OK = 0,
    MHA_ERR_INVALID_ARG = 1,   /* bad size, null required pointer, small workspace */
    MHA_ERR_UNSUPPORTED = 2,   /* valid per the pages but not implemented (e.g. d_k > 256) */
    MHA_ERR_CUDA = 3           /* a CUDA call failed; see mha_last_error() */
} mha_status_t;

typedef enum { MHA_F32 = 0, MHA_BF16 = 1 } mha_dtype_t;

typedef struct {
    int causal;                     /* nonzero: subsequent mask, key j <= query i */
    const int32_t* key_valid_lens;  /* device [B] or NULL: key j allowed iff j < len[b]; len < 0 reads as 0 */
    const uint8_t* dense;           /* device [B, dense_mq, L_k] or NULL: 0 = masked */
    int dense_mq;                   /* 1 (broadcast over queries) or L_q; ignored if dense is NULL */
} mha_mask_t;

/*
 * Workspace the forward pass needs, in bytes (a multiple of 256).
 * Layout (each part starts on a 256-byte boundary, element type = dt):
 *   Qh   [B, h, L_q, d_k]      head-split projected queries
 *   KVh  [B, 2, h, L_k, d_k]   head-split projected keys (slot 0) and values (slot 1)
 *   ctx  [B, L_q, d_model]     concatenated head outputs (input of W_o)
 *   stat [B, h, L_q, 2] fp32   per-row softmax statistics (max, sum) used for p_attn
 *   sched 256 bytes            2 ints: the d_k = 128 attention's work counter (zeroed by the
 *                              Q/K/V projection stage, left at zero by the attention stage)
 * For MHA_BF16 with a d_k the tensor-core kernels do not take (d_k <= 256): the MHA_F32
 * workspace of the same sizes, then fp32 copies of query, key, value [B, L, d_model], of
 * the four weights and biases and of out, each 256-byte aligned.
 * Returns 0 for invalid sizes.
 */
size_t mha_workspace_size(mha_dtype_t dt, int B, int L_q, int L_k, int d_model, int h);

/*
 * mha_forward -- the whole sublayer: out = MultiHeadedAttention(query, key, value, mask).
 *   query [B, L_q, d_model]; key, value [B, L_k, d_model]   (may alias each other)
 *   w_q, w_k, w_v, w_o [d_model, d_model] stored (out, in); b_* [d_model] or NULL (= zero bias)
 *   mask   NULL = no mask
 *   out    [B, L_q, d_model], type dt; must not alias any input or the workspace
 *   p_attn NULL, or fp32 [B, h, L_q, L_k]: the attention weights of every head
 *          (the pages keep them as self.attn for visualisation)
 *   workspace >= mha_workspace_size(...) bytes of device memory, 256-byte aligned
 * Three stages run in order on `stream`: mha_qkv_projection, mha_attention_core,
 * mha_output_projection.
 */
mha_status_t mha_forward(mha_dtype_t dt,
                         const void* query, const void* key, const void* value,
                         const void* w_q, const void* b_q,
                         const void* w_k, const void* b_k,
                         const void* w_v, const void* b_v,
                         const void* w_o, const void* b_o,
                         int B, int L_q, int L_k, int d_model, int h,
                         const mha_mask_t* mask,
                         void* out, float* p_attn,
                         void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * Stage 1 -- the three input projections of MultiHeadedAttention.forward, written
 * head-split into the workspace (Qh and KVh above). One launch covers all three.
 */
mha_status_t mha_qkv_projection(mha_dtype_t dt,
                                const void* query, const void* key, const void* value,
                                const void* w_q, const void* b_q,
                                const void* w_k, const void* b_k,
                                const void* w_v, const void* b_v,
                                int B, int L_q, int L_k, int d_model, int h,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stage 2 -- attention() for every (batch, head): scores, scale, -1e9 fill,
 * softmax, P.V, written concatenated into ctx of the workspace; and, if p_attn
 * is not NULL, the normalised weights fp32 [B, h, L_q, L_k]. Reads Qh and KVh.
 */
mha_status_t mha_attention_core(mha_dtype_t dt, int B, int L_q, int L_k, int d_model, int h,
                                const mha_mask_t* mask, float* p_attn,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stage 3 -- the fourth Linear of MultiHeadedAttention: out = ctx W_o^T + b_o,
 * reading ctx from the workspace. out [B, L_q, d_model], type dt.
 */
mha_status_t mha_output_projection(mha_dtype_t dt, const void* w_o, const void* b_o,
                                   int B, int L_q, int L_k, int d_model, int h,
                                   void* out, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * mha_forward_host -- the same sublayer with the activations in HOST memory:
 * query/key/value are read from host buffers and out is written to a host
 * buffer; weights, biases, mask parts and the workspace are device pointers as
 * above. The host buffers should be page-locked for the copies to be
 * asynchronous. `staging` is device memory of at least
 * mha_host_staging_size(...) bytes that receives the activations. The call is
 * pipelined over chunks of sequences (up to 4 when query, key and value hold
 * at least 32 MiB of host data together, else up to 2; never more than B) with
 * library-owned streams (one set
 * per device, created on first use): an upload stream, a download stream and a
 * second compute stream. Chunks alternate between `stream` and the second
 * compute stream when the workspace holds two chunk workspaces (each
 * mha_workspace_size(dt, ceil(B / chunks), ...) bytes; true whenever B >= 2 at
 * realistic sizes), otherwise all run on `stream`. When query, key and value
 * are the same host buffer (bf16, L >= 256), the first chunk is uploaded and
 * projected in two row windows and the last chunk's output projection and
 * download run in two row windows. Copies: host->device of query (and of key and value unless they
 * alias query / each other), device->host of out; all ordered by events. When
 * the call returns, all of it is enqueued behind `stream`: synchronise `stream`
 * before reading out. The workspace must not be used by other work on other
 * streams while the call runs.
 */
size_t mha_host_staging_size(mha_dtype_t dt, int B, int L_q, int L_k, int d_model,
                             int kv_distinct, int q_distinct);
mha_status_t mha_forward_host(mha_dtype_t dt,
                              const void* h_query, const void* h_key, const void* h_value,
                              const void* w_q, const void* b_q,
                              const void* w_k, const void* b_k,
                              const void* w_v, const void* b_v,
                              const void* w_o, const void* b_o,
                              int B, int L_q, int L_k, int d_model, int h,
                              const mha_mask_t* mask,
                              void* h_out,
                              void* staging, size_t staging_bytes,
                              void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * mha_forward_noalloc -- mha_forward for callers that cannot allocate device
 * memory. (The pages have no counterpart: this is an interface choice of this
 * library.) Some callers are handed only their inputs and outputs: a plugin
 * whose host application owns all device memory through its own pool, a
 * serving path that must never hit cudaMalloc (which can synchronise the whole
 * device), an interface with no workspace argument. This entry point takes the
 * same arguments as mha_forward minus the workspace, allocates nothing, and
 * uses a fixed scratch area built into the library instead:
 *   - MHA_NOALLOC_SCRATCH_BYTES (48 MiB) of device memory, reserved on every
 *     GPU that loads this part of the library and held until the process exits.
 *   - Problems whose mha_workspace_size(...) exceeds it are rejected with
 *     MHA_ERR_INVALID_ARG and a message naming both sizes (e.g. the encoder,
 *     decoder and cross-attention workloads of this library fit; B=4, L=8192,
 *     d_model=1024 does not).
 *   - The first call on each device looks up the scratch address with that
 *     device current; make that first call before any stream capture begins.
 *     The address belongs to the device's current CUDA context: after the
 *     context is destroyed and re-created (e.g. cudaDeviceReset), the next
 *     call sees the new context and looks the address up again, so that call
 *     too belongs outside stream capture.
 *   - All calls on a device share the one scratch area: calls whose work
 *     overlaps on the GPU (other streams, other host threads) race and corrupt
 *     each other. Serialise them, e.g. on one stream.
 *   - Nothing in the scratch needs to start at zero; it is not cleared.
 */
#define MHA_NOALLOC_SCRATCH_BYTES ((size_t)48 << 20)
mha_status_t mha_forward_noalloc(mha_dtype_t dt,
                                 const void* query, const void* key, const void* value,
                                 const void* w_q, const void* b_q,
                                 const void* w_k, const void* b_k,
                                 const void* w_v, const void* b_v,
                                 const void* w_o, const void* b_o,
                                 int B, int L_q, int L_k, int d_model, int h,
                                 const mha_mask_t* mask,
                                 void* out, float* p_attn,
                                 void* stream);

/*
 * The residual sublayer around multi-head attention, pre-norm form
 * ("The Annotated Transformer", SublayerConnection: x + dropout(sublayer(norm(x))),
 * dropout = identity):
 *   y   = LayerNorm(x)
 *   out = x + MultiHeadedAttention(y, y, y, mask)              if memory == NULL (self-attention)
 *   out = x + MultiHeadedAttention(y, memory, memory, mask)    otherwise (source attention,
 *         "The Annotated Transformer", DecoderLayer: src_attn(x, m, m, src_mask))
 * LayerNorm over the last dimension, ln_kind selects the pages' two forms:
 *   0  a (x - mean) / (std + eps) + b, std unbiased ("The Annotated Transformer", LayerNorm, eps 1e-6)
 *   1  a (x - mean) / sqrt(var + eps) + b, var biased (nn.LayerNorm, "003-Transformer")
 *   ln_gain / ln_bias [d_model] or NULL (ones / zeros), type dt.
 * x [B, L, d_model]; memory [B, L_mem, d_model] or NULL; out [B, L, d_model] (may alias x: each
 * element of x is read by the thread that then writes the same element of out).
 * d_model <= 2048. Workspace >= mha_sublayer_workspace_size(...): LayerNorm(x) followed by the
 * workspace of mha_forward. Launches: LayerNorm, the three stages of mha_forward, with the
 * residual added in the W_o epilogue.
 */
size_t mha_sublayer_workspace_size(mha_dtype_t dt, int B, int L, int L_mem, int d_model, int h);
mha_status_t mha_sublayer_forward(mha_dtype_t dt, const void* x, const void* memory,
                                  const void* ln_gain, const void* ln_bias, float ln_eps, int ln_kind,
                                  const void* w_q, const void* b_q,
                                  const void* w_k, const void* b_k,
                                  const void* w_v, const void* b_v,
                                  const void* w_o, const void* b_o,
                                  int B, int L, int L_mem, int d_model, int h,
                                  const mha_mask_t* mask,
                                  void* out, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * Incremental decoding with a key/value cache (bf16, d_k = 64 or 128).
 * At prediction time the d2l Transformer decoder (d2l Transformer chapter, DecoderBlock:
 * state[2] keeps the representations decoded so far and torch.cat appends the new one as
 * keys and values) attends from the newest token to every token so far, itself included.
 * This library caches the PROJECTED keys and values, which gives the same result.
 *   k_cache, v_cache  device [B, h, L_max, d_k] bf16: position t of sequence b, head i.
 *   mha_kv_cache_prefill: projects x [B, T, d_model] into positions 0..T-1 of both caches
 *     (K = x W_k^T + b_k, V = x W_v^T + b_v); T <= L_max.
 *   mha_decode_step: one new token per sequence, x_new [B, d_model]:
 *     q, k, v = x_new W^T + b; k, v written at position cache_len[b] (device int32 [B]),
 *     which the step then increments on the device; out [B, d_model] = the sublayer's output
 *     for the new token: attention of q over the cache_len[b] + 1 cached positions (no mask
 *     needed), concat, W_o. A sequence whose cache is full (cache_len[b] >= L_max) appends
 *     nothing and the step records code 0x301 in the device status word
 *     (mha_check_device_status). Workspace >= mha_decode_workspace_size(...), 256-byte aligned.
 */
size_t mha_decode_workspace_size(int B, int d_model, int h, int L_max);
mha_status_t mha_kv_cache_prefill(mha_dtype_t dt, const void* x,
                                  const void* w_k, const void* b_k,
                                  const void* w_v, const void* b_v,
                                  int B, int T, int d_model, int h,
                                  void* k_cache, void* v_cache, int L_max, void* stream);
mha_status_t mha_decode_step(mha_dtype_t dt, const void* x_new,
                             const void* w_q, const void* b_q,
                             const void* w_k, const void* b_k,
                             const void* w_v, const void* b_v,
                             const void* w_o, const void* b_o,
                             int B, int d_model, int h,
                             void* k_cache, void* v_cache, int32_t* cache_len, int L_max,
                             void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Position-wise feed-forward network ("003-Transformer" tutorial, feed-forward
 * layer; "From RNN to Attention", part 3, FFN):
 *   out = max(0, x W_1^T + b_1) W_2^T + b_2        (dropout = identity)
 *   x [B, L, d_model]; w_1 [d_ff, d_model], b_1 [d_ff] or NULL;
 *   w_2 [d_model, d_ff], b_2 [d_model] or NULL; out [B, L, d_model], type dt.
 *   MHA_BF16: d_model and d_ff multiples of 64, 16-byte aligned pointers; the
 *   two layers run on the tensor-core GEMM (ReLU fused into the first epilogue).
 *   The hidden activations [B, L, d_ff] live in the caller's workspace of at
 *   least mha_ffn_workspace_size(...) bytes (256-byte aligned).
 */
size_t mha_ffn_workspace_size(mha_dtype_t dt, int B, int L, int d_model, int d_ff);
mha_status_t mha_ffn_forward(mha_dtype_t dt, const void* x,
                             const void* w_1, const void* b_1,
                             const void* w_2, const void* b_2,
                             int B, int L, int d_model, int d_ff,
                             void* out, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * ======================================================================================
 * Serving operators: rotary positions, a paged key/value cache (also in 8 bits) and its block table, attention over it, attention
 * with capped and biased scores under span masks, RMS norm with 8-bit output.
 *
 * Tensors here need not be contiguous: a [B, L, heads, d_k] tensor is a pointer and the three
 * strides below, in elements; the d_k elements of one head are adjacent. So the same call takes
 * [B, L, h, d_k], the workspace's [B, h, L, d_k], and slices of one packed projection. Strides
 * may be 0 in an input (a broadcast); outputs must not overlap themselves. Offsets are 64-bit.
 * Pointers are aligned to their element type; where a call needs more it says so.
 * ======================================================================================
 */
typedef struct {
    int64_t b, l, h;
} mha_strides_t;

/*
 * Rotary positions. The first rot_dim features of a head form rot_dim / 2 pairs (x_0, x_1):
 * features (i, i + rot_dim / 2) in the half layout, (2 i, 2 i + 1) interleaved. A token at
 * position t turns pair i by the angle t * inv_freq[i]:
 *   (x_0, x_1) -> scale * (x_0 cos - x_1 sin, x_1 cos + x_0 sin)
 * Features rot_dim .. d_k - 1 pass unchanged. The angle is formed to about 2^-46 of its size and
 * reduced before it is rounded, so positions up to 2^24 keep fp32 accuracy (beyond, the error of cos and sin grows
 * with the position: 2^-17.5 at 2^29); products are in fp32, rounded once to the type of the tensor.
 */
typedef struct {
    const float* inv_freq;   /* device fp32 [rot_dim / 2] */
    int rot_dim;             /* even, 2 <= rot_dim <= d_k */
    int interleaved;         /* 0: half layout, 1: interleaved pairs */
    float scale;             /* multiplies cos and sin (1: none) */
} mha_rotary_t;

/*
 * Host helper: fills inv_freq (HOST memory, rot_dim / 2 floats) and *scale for a context scaled by
 * `factor` against the `original_length` that the model was trained with.
 *   MHA_ROPE_PLAIN   base^(-2 i / rot_dim)
 *   MHA_ROPE_LINEAR  plain / factor (positions interpolated)
 *   MHA_ROPE_BASE    plain with base * factor^(rot_dim / (rot_dim - 2)) (the base stretched)
 *   MHA_ROPE_BANDED  by wavelength w = 2 pi / f: kept below original_length / high, divided by
 *                    factor above original_length / low, a blend linear in original_length / w between
 *   MHA_ROPE_RAMP    by index: kept up to the pair that turns `high` times over original_length,
 *                    divided by factor from the one that turns `low` times, linear in the index
 *                    between (indices rounded outwards, limited to 0 .. rot_dim - 1);
 *                    *scale = 0.1 ln(factor) + 1
 * *scale is 1 for the others. low < high; both ignored by the first three.
 */
typedef enum {
    MHA_ROPE_PLAIN = 0, MHA_ROPE_LINEAR = 1, MHA_ROPE_BASE = 2, MHA_ROPE_BANDED = 3, MHA_ROPE_RAMP = 4
} mha_rope_scaling_t;
mha_status_t mha_rotary_frequencies(float* inv_freq, float* scale, int rot_dim, double base,
                                    mha_rope_scaling_t scaling, double factor, double original_length,
                                    double low, double high);

/*
 * Turns queries and keys: q [B, T, h, d_k] -> q_out, and, unless k is NULL, k [B, T, h_kv, d_k] ->
 * k_out. positions: device int32 [B, T] (any value, contiguous) or NULL for 0 .. T-1. An output may
 * be its input with the same strides (in place); otherwise they must not overlap. MHA_F32 or MHA_BF16,
 * any d_k <= 512. h_kv, the k strides and k_out are ignored if k is NULL. One launch.
 */
mha_status_t mha_rotary(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                        void* q_out, const mha_strides_t* q_out_strides,
                        const void* k, const mha_strides_t* k_strides,
                        void* k_out, const mha_strides_t* k_out_strides,
                        int B, int T, int h, int h_kv, int d_k, const int32_t* positions,
                        const mha_rotary_t* rotary, void* stream);

/*
 * A paged key/value cache: n_pages pages of page_size slots, each slot h_kv heads of d_k, in two
 * arrays with the same strides (in elements; d_k adjacent). Position t of sequence b lives in slot
 * t % page_size of page block_table[b * table_stride + t / page_size]; max_pages entries of a row
 * are read at most, so a sequence holds up to max_pages * page_size positions. Any page_size >= 1.
 * Pages that a call writes must be distinct between (and within) sequences; pages only read may be
 * shared. A page number outside [0, n_pages), or a position beyond the table, is never followed:
 * the append skips the token, the attention leaves the position out (a length beyond the table is
 * cut to it), and both record MHA_PAGED_BAD_PAGE in the device status word.
 */
typedef struct {
    void* k_pages;
    void* v_pages;
    int64_t page_stride, slot_stride, head_stride;
    int n_pages, page_size;
    const int32_t* block_table;
    int64_t table_stride;
    int max_pages;
} mha_paged_cache_t;
#define MHA_PAGED_BAD_PAGE 0x501

/*
 * Appends T new tokens a sequence to the cache and turns queries and keys on the way, in one launch.
 *   k, v [B, T, h_kv, d_k]; start: device int32 [B], the positions already held (token t of
 *   sequence b goes to position start[b] + t, which is also its rotary position);
 *   new_lens: device int32 [B] or NULL: only tokens t < new_lens[b] exist; the rest is not read and
 *   their outputs are left as they were; rotary NULL: keys enter as they are.
 *   k_out NULL, or [B, T, h_kv, d_k]: the turned keys, for an attention over the prompt itself.
 *   q NULL, or [B, T, h, d_k] -> q_out turned the same way.
 * In-place rules as for mha_rotary; no output overlaps another input either (k_out may be k only
 * where v is not the same memory). start is not changed: the caller adds the counts.
 */
mha_status_t mha_paged_append(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                              void* q_out, const mha_strides_t* q_out_strides,
                              const void* k, const mha_strides_t* k_strides,
                              void* k_out, const mha_strides_t* k_out_strides,
                              const void* v, const mha_strides_t* v_strides,
                              int B, int T, int h, int h_kv, int d_k, const int32_t* start,
                              const int32_t* new_lens, const mha_rotary_t* rotary,
                              const mha_paged_cache_t* cache, void* stream);

/*
 * How a score is formed from q . k:
 *   s = scale * q.k;  cap > 0: s = cap * tanh(s / cap);  slopes: s -= slopes[head] * |i - j|
 * with i, j the positions of the query and the key.
 */
typedef struct {
    float scale;             /* 0: 1 / sqrt(d_k) */
    float cap;               /* 0: no cap; scale / cap finite. Taken as 2^-100 or 2^100 beyond them */
    const float* slopes;     /* device fp32 [h] or NULL */
} mha_scores_t;

/*
 * Attention of one new token a sequence over the paged cache:
 *   out[b, i] = sum_j softmax_j(s)[j] v[j, i / (h / h_kv)],  j = 0 .. kv_lens[b] - 1
 * for the query q [B, h, d_k] at position kv_lens[b] - 1 (append its key and value first). q and out
 * have strides (b, h; l is ignored). kv_lens: device int32 [B]; a length <= 0 gives zeros. scores NULL:
 * the plain scaled scores. MHA_BF16 or MHA_F32, d_k = 64 or 128, h a multiple of h_kv. What lies in a
 * page behind a sequence's end is not used, whatever it holds. The pages and their strides are aligned
 * to 16 bytes. Weights enter the product with bf16 values as two bf16 terms: the result is within its own rounding.
 * workspace >= mha_paged_attention_workspace_size(...), 256-byte aligned, contents of no matter;
 * calls that overlap on the GPU need one each. The result does not depend on timing.
 */
size_t mha_paged_attention_workspace_size(mha_dtype_t dt, int B, int h, int h_kv, int d_k);
mha_status_t mha_paged_attention(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                                 void* out, const mha_strides_t* out_strides,
                                 int B, int h, int h_kv, int d_k, const int32_t* kv_lens,
                                 const mha_scores_t* scores, const mha_paged_cache_t* cache,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * The block table of a paged cache as sequences grow, shrink and end, on the device: sequence b goes from held[b] to want[b]
 * positions (device int32 [B], B <= 2^24; below 0: 0), so from ceil(held / page_size) to ceil(want / page_size) pages.
 *   free_pages  device int32 [n_pages], a stack: entries 0 .. *free_count - 1 are the free pages; the two are updated.
 *   Sequences that shrink (want 0: end) give their last pages back: entry by entry pushed so that the first sequence's first
 *   page ends on top, and -1 in the table. Then those that grow take pages from the top in the order of the sequences, the first
 *   one's first, and find them in the table. Pages given back in a call serve in the same call.
 *   Served is a sequence that needs no page, or whose pages and those of all sequences before it are there; one that
 *   is not, or that wants more than max_pages pages, stays as it is.
 *   lens      device int32 [B]: positions after the call: want[b], or held[b] where it is not served.
 *   new_lens  device int32 [B] or NULL: max(lens - held, 0), for the append (with start = held).
 *   slots     device int64 [B, T] or NULL: of new token t of sequence b, page * page_size + slot in the page, -1 where there is
 *             none (t >= new_lens[b]). T is ignored without it.
 * A call with held and want exchanged takes a step back, the stack included. Entries of the table that a call does not name, and
 * of the stack above the pages given back, are left as they were. A page number outside [0, n_pages) moves as it is, gives no slot
 * and records MHA_PAGED_BAD_PAGE, and so does a stack that pages given back would overflow (the ones beyond n_pages are
 * dropped). lens and new_lens overlap neither held nor want nor each other. Calls that share a table or a stack are ordered by the caller.
 * A page has one owner: it stands once among the rows' held pages and the free ones, and that is not looked at. A page of several rows (a
 * common prefix, which the attention reads as any other) would be given back by each of them and then granted twice; of whole pages that are
 * shared, give the call the table's columns behind them, and held and want without their positions.
 */
mha_status_t mha_paged_resize(const int32_t* held, const int32_t* want, int B, int page_size,
                              int32_t* block_table, int64_t table_stride, int max_pages,
                              int32_t* free_pages, int n_pages, int32_t* free_count,
                              int32_t* lens, int32_t* new_lens, int T, int64_t* slots, void* stream);

/*
 * A paged cache in 8 bits: pages as above, strides in codes (bytes), d_k = 64 or 128; each block of `block` neighbouring
 * slots of a page and each key head has a scale for keys and one for values, and a code c stands for c * scale.
 */
typedef enum { MHA_CODE_E4M3 = 0, MHA_CODE_INT8 = 1 } mha_code_t;   /* e4m3: finite form, NaN; int8: two's complement */
typedef struct {
    mha_paged_cache_t pages;   /* pages and strides aligned to 16 bytes */
    mha_code_t code;
    int block;                 /* tokens that a scale covers: divides page_size; up to 256 for the append */
    float* k_scales;           /* device fp32 [n_pages, page_size / block, h_kv], contiguous, below 2^31 a page */
    float* v_scales;
} mha_coded_cache_t;

/*
 * mha_paged_append into such a cache. The scale of a block is the smallest power of two s, at least 2^-120, with
 * max |x| <= top * s over the turned keys (the values) of its tokens, top = 448 (e4m3) or 127 (int8), x in fp32; codes are
 * x / s rounded to nearest even. A token at a block's first slot begins the block: what its scale and slots held is forgotten.
 * Tokens that enter a block behind others keep the block's scale if theirs is not larger; else the block gets theirs, and the codes
 * in front of them are rounded again (c * old / new). A scale of other origin is kept as it is while it is the larger one.
 * A NaN or an infinity makes its block's scale NaN, and with it whatever attends to the block.
 *   q, k, v, q_out, k_out: pointers and strides aligned to 16 bytes; k_out gets the turned keys in type dt. Otherwise all
 * is as for mha_paged_append: start, new_lens, rotary, in-place rules, bad pages. Blocks are written by one sequence each. One launch.
 */
mha_status_t mha_coded_append(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                              void* q_out, const mha_strides_t* q_out_strides,
                              const void* k, const mha_strides_t* k_strides,
                              void* k_out, const mha_strides_t* k_out_strides,
                              const void* v, const mha_strides_t* v_strides,
                              int B, int T, int h, int h_kv, int d_k, const int32_t* start,
                              const int32_t* new_lens, const mha_rotary_t* rotary,
                              const mha_coded_cache_t* cache, void* stream);

/*
 * mha_paged_attention over such a cache: the attention over the values c * scale, for q and out of type dt. Scales are
 * 0 or between 2^-120 and 2^122, of any mantissa, and |c * scale| of the values sums to less than 2^120 over a sequence. q enters as it is (bf16: exact down to 2^-29 of its row's largest element; fp32:
 * to 2^-22 of itself or 2^-39 of that); weights (a softmax numerator times its value's scale) are rounded to 2^-11 of themselves or 2^-35 of the row's
 * largest for a bf16 result, to 2^-22 or 2^-47 for an fp32 one (the second bounds where the largest's scale is from 2^-106 to 2^112, and rising
 * to 2^-21 and 2^-33 at 2^-120, 2^-38 at 2^122); products and sums are fp32. A key whose softmax numerator is below 2^-126 of the row's largest may
 * count as none, whatever the scale of its value.
 * What lies behind a sequence's end is not used; a block's scale is, for the block's other slots.
 * workspace >= mha_coded_attention_workspace_size(...); kv_lens, scores, bad pages, order: as for mha_paged_attention.
 */
size_t mha_coded_attention_workspace_size(mha_dtype_t dt, int B, int h, int h_kv, int d_k);
mha_status_t mha_coded_attention(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                                 void* out, const mha_strides_t* out_strides,
                                 int B, int h, int h_kv, int d_k, const int32_t* kv_lens,
                                 const mha_scores_t* scores, const mha_coded_cache_t* cache,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * The keys that a query may attend to, as the intersection of (all optional):
 *   causal          key j <= q_offset + i, or j < prefix_lens[b] (a prefix that all may see)
 *   key_valid_lens  key j < key_valid_lens[b]
 *   doc_spans       doc_spans[b, i, 0] <= key j < doc_spans[b, i, 1] (mha_document_spans)
 * Query i has position q_offset + i. A query without any key gives a row of zeros (not the uniform
 * row of mha_forward's -1e9 fill).
 */
typedef struct {
    int causal;
    int q_offset;                   /* >= 0: keys before the first query, L_k - L_q where both end together */
    const int32_t* key_valid_lens;  /* device [B] or NULL */
    const int32_t* prefix_lens;     /* device [B] or NULL; read only if causal */
    const int32_t* doc_spans;       /* device [B, L_q, 2] or NULL */
} mha_span_mask_t;

/*
 * spans[b, i] = [first, last + 1) of the run of equal doc_ids around position i; (0, 0) where
 * doc_ids < 0 (padding). doc_ids, device int32 [B, L]: each document is one run. spans: device
 * int32 [B, L, 2]. Serves every layer of a batch.
 */
mha_status_t mha_document_spans(const int32_t* doc_ids, int B, int L, int32_t* spans, void* stream);

/*
 * Attention with grouped heads over strided tensors, scores and mask as above:
 *   q [B, L_q, h, d_k], k and v [B, L_k, h_kv, d_k] -> out [B, L_q, h, d_k]
 * h a multiple of h_kv (head n reads key head n / (h / h_kv)); scores, mask NULL: plain, all keys.
 * MHA_BF16 or MHA_F32 with d_k = 64 or 128; pointers and strides aligned to 16 bytes. Keys and values at and
 * behind key_valid_lens[b] are not used, whatever they hold; elsewhere a masked value that is not
 * finite may reach rows that do not attend to it (0 * NaN), but no row without a key. Weights are rounded to bf16
 * for the product with bf16 values. The l stride of q, k and v is not 0 (unless the length is 1). No workspace.
 */
mha_status_t mha_attention(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides,
                           const void* k, const mha_strides_t* k_strides,
                           const void* v, const mha_strides_t* v_strides,
                           void* out, const mha_strides_t* out_strides,
                           int B, int L_q, int L_k, int h, int h_kv, int d_k,
                           const mha_scores_t* scores, const mha_span_mask_t* mask, void* stream);

/*
 * RMS norm of rows, with the residual's addition before it and, on request, 8-bit output:
 *   z = x + residual;  y = gain * z / sqrt(mean(z^2) + eps)
 *   x, residual, sum [rows, d] with row strides (elements), type dt; residual NULL: z = x, and sum is
 *   ignored; sum NULL: z is not written. sum may be x or residual, and y of type dt too if sum is not (same
 *   stride). The norm is of the fp32 sum, not of its rounding. gain [d] type dt, or NULL (ones).
 *   scales NULL: y has type dt. Otherwise y is e4m3 (1 byte an element, finite form): each group of
 *   `group` elements of a row (0: the whole row; else 32, 64 or 128, dividing d) has
 *   scale = max |y| / 448 (1 where that is 0) to within 2^-23, y8 = y / scale rounded to nearest even, and scales
 *   [rows, groups], fp32, contiguous, receives it. NaN stays NaN.
 *   1 <= d <= 2^30; rows >= 0. The squares are summed in fp32: their sum has to stay below 2^128, and values below
 *   2^-63 lose digits in it.
 */
mha_status_t mha_rmsnorm(mha_dtype_t dt, const void* x, int64_t x_stride, const void* residual,
                         int64_t residual_stride, void* sum, int64_t sum_stride, const void* gain, float eps,
                         int64_t rows, int d, void* y, int64_t y_stride, float* scales, int group, void* stream);

/* Message for the last non-OK status returned on this thread ("" if none). */
const char* mha_last_error(void);

/*
 * Device-side status of the bounded waits inside the tensor-core kernels.
 * Every pipeline wait gives up after a fixed iteration budget instead of
 * spinning forever; when one gives up, the kernel records a code here and runs
 * to completion (its outputs are then not valid). This call SYNCHRONISES the
 * device, copies the word to *status (0 = no wait gave up), and, if reset is
 * nonzero, clears it.
 */
mha_status_t mha_check_device_status(int* status, int reset);

/*
 * Diagnostic: exercises the failure path of the bounded pipeline waits on the GPU.
 * Enqueues on `stream` one warp that waits on an mbarrier nothing ever arrives on,
 * through the same bounded wait every tensor-core pipeline uses but with a budget of
 * 1024 rounds; the wait gives up, the kernel records MHA_SELFTEST_WAIT_CODE in the
 * device status word (unless a code is already there) and ends. Read the word with
 * mha_check_device_status. Nothing faults, traps or hangs, and no other work of the
 * library is affected.
 */
#define MHA_SELFTEST_WAIT_CODE 0x7f1
mha_status_t mha_selftest_wait_timeout(void* stream);

/* Library version string. */
const char* mha_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GB300_MHA_H */
