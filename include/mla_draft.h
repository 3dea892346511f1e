/*
 * mla_draft.h -- C ABI of the MLA (Multi-head Latent Attention) draft-layer
 * forward for NVIDIA GB300 (sm_103a).
 *
 * What the layer computes (sources are web pages, cited by title/section):
 *  - "MLA (Multi-Head Latent Attention)" blog, DeepseekV2MLAAttention.__init__
 *    and MultiHeadLatentAttentionWrapper.forward: optional low-rank query
 *    (fused_qkv_a_proj -> q_a_layernorm -> q_b_proj, or q_proj without
 *    q_lora_rank), the shared compressed KV latent (kv_a_proj_with_mqa ->
 *    kv_a_layernorm), partial RoPE on qk_rope_head_dim, kv_b_proj expansion,
 *    o_proj.
 *  - same blog, do_kv_cache_update / concat_and_cache_mla and
 *    get_kv_cache_shape: the latent cache [num_pages, page_size,
 *    kv_lora_rank + qk_rope_head_dim], one entry [kv_c_normed | k_pe] per
 *    token, written by slot index.
 *  - same blog, forward_impl (MQA branch) and forward_mqa: attention in the
 *    latent space (q_nope @ W_UK, scores against [c | k_pe], W_UV up-proj).
 *  - "Add config-selectable MLA draft attention" (SpecForge PR #758),
 *    Summary/Structure: DFlash-family target-context injection, full/sliding
 *    masks, zeroing of fully masked queries, optional output gate, NeoX or
 *    interleaved rotation; dimension validation once at init.
 *  - "extract GQA/MLA attention into reusable layers" (SpecForge PR #1026),
 *    Modifications: masks by logical position; empty queries zeroed before
 *    o_proj.
 *
 * Conventions for every entry point
 *  - Pointers named "device" are CUDA device pointers (cudaMalloc / torch),
 *    "host" pointers are CPU memory.  The library never allocates device
 *    memory: weights, arena, cache, workspace and outputs belong to the
 *    caller.  The library owns only the host-side handle.
 *  - Weights use torch.nn.Linear layout W[out, in], row-major, contiguous, of
 *    the config's dtype (bf16 or fp32).  Hidden states are row-major
 *    [tokens, hidden_size] of the same dtype; so is the cache.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  append and
 *    forward only enqueue work: no host synchronisation, no allocation.
 *  - Errors: host-side validation returns a status and never aborts; the
 *    message is available from mla_last_error().  Index errors found on the
 *    device (slot, page or position out of range) skip the offending access
 *    and set a bit in a device status word read by mla_get_device_status().
 *  - Devices: one GPU per process.  A handle works on the device that was
 *    current at mla_draft_init, which must be current for every call; the
 *    library keeps per-process launch settings (kernel shared-memory limits,
 *    the SM count and cluster occupancy) taken from the first device it
 *    runs on.  The multi-GPU model is one process per GPU.
 */
#ifndef MLA_DRAFT_H
#define MLA_DRAFT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t mla_status_t;
enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, inconsistent dims    */
  MLA_ERR_UNSUPPORTED = 2,   /* valid dims this build has no kernel for       */
  MLA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed             */
  MLA_ERR_DEVICE_CHECK = 4,  /* the device reported an index error            */
  MLA_ERR_TIMEOUT = 5        /* a bounded device wait expired                 */
};

enum { MLA_BF16 = 0, MLA_FP32 = 1,                /* mla_config_t.dtype */
       MLA_FP16 = 2 };                            /* probabilities only (mla_verify_drafts) */
enum { MLA_ROPE_NEOX = 0, MLA_ROPE_INTERLEAVED = 1 }; /* mla_config_t.rope */

/* Bits of the device status word (mla_get_device_status). */
enum {
  MLA_DEV_BAD_SLOT = 1,      /* slot_mapping entry outside the cache          */
  MLA_DEV_BAD_POSITION = 2,  /* position < 0 or >= max_position               */
  MLA_DEV_BAD_PAGE = 4,      /* block_table entry outside [0, num_pages)      */
  MLA_DEV_TIMEOUT = 8,       /* a bounded mbarrier wait gave up               */
  MLA_DEV_BAD_LENGTH = 16,   /* kv_len < 0 or > max_pages * page_size         */
  MLA_DEV_BAD_WINDOW = 32,   /* window < 0 (the block's rows are zeroed)      */
  MLA_DEV_BAD_TREE = 64,     /* a node's parent is not an earlier node        */
  MLA_DEV_BAD_KEEP = 128,    /* a list of kept keys that is not ascending in
                                [0, kv_len), or longer than its sequence      */
  MLA_DEV_BAD_DRAFT = 256,   /* a drafted token outside the vocabulary, or a
                                row of the target without any mass            */
  MLA_DEV_BAD_SCALE = 512    /* a scale of an 8-bit cache that is no power of
                                two (its readers become NaN)                  */
};

/* Intermediate tensors the forward leaves in its workspace
 * (mla_forward_workspace_offset). */
enum { MLA_WS_Q_ABS = 0, MLA_WS_O_LAT = 1, MLA_WS_O = 2, MLA_WS_LSE = 3 };

/* Layer configuration.  Structural dims follow the HF DeepSeek-V2/V3 fields;
 * q_lora_rank == 0 selects the non-low-rank path (q_proj +
 * kv_a_proj_with_mqa).  softmax_scale == 0 means 1/sqrt(qk_nope + qk_rope).
 * max_position bounds the RoPE table built at init. */
typedef struct {
  int32_t hidden_size, num_heads, q_lora_rank, kv_lora_rank;
  int32_t qk_nope_head_dim, qk_rope_head_dim, v_head_dim;
  int32_t rope;              /* MLA_ROPE_NEOX | MLA_ROPE_INTERLEAVED          */
  int32_t use_output_gate;   /* 0/1: o *= sigmoid(x @ gate_proj^T)            */
  int32_t dtype;             /* MLA_BF16 | MLA_FP32                           */
  int32_t page_size;         /* tokens per cache page                         */
  int32_t max_position;      /* positions must lie in [0, max_position)       */
  double rope_theta, rms_norm_eps, softmax_scale;
} mla_config_t;

/* Device pointers to the layer's parameters, read only inside mla_draft_init
 * (not retained).  Unused fields are NULL. */
typedef struct {
  const void *fused_qkv_a_proj;    /* [q_lora_rank + kv_lora_rank + qk_rope, D]  (q_lora_rank > 0) */
  const void *q_a_layernorm;       /* [q_lora_rank]                               (q_lora_rank > 0) */
  const void *q_b_proj;            /* [H * (qk_nope + qk_rope), q_lora_rank]      (q_lora_rank > 0) */
  const void *q_proj;              /* [H * (qk_nope + qk_rope), D]                (q_lora_rank == 0) */
  const void *kv_a_proj_with_mqa;  /* [kv_lora_rank + qk_rope, D]                 (q_lora_rank == 0) */
  const void *kv_a_layernorm;      /* [kv_lora_rank]                                                */
  const void *kv_b_proj;           /* [H * (qk_nope + v_head), kv_lora_rank]                        */
  const void *gate_proj;           /* [H * v_head, D]                             (use_output_gate) */
  const void *o_proj;              /* [D, H * v_head]                                               */
} mla_weights_t;

/* Which keys each query block attends (device pointers).  Block b holds
 * queries b*block_len .. (b+1)*block_len-1.  Its key j (logical position j)
 * is the cache entry at page block_table[b*max_pages + j/page_size], row
 * j%page_size.  Key j is visible to query i of block b iff
 *   q_visible[i] != 0  &&  j < kv_len[b]  &&
 *   (window[b] == 0 || positions[i] - j < window[b]).
 * A query with no visible key produces an exact zero output row.  A negative
 * window is rejected on the device: MLA_DEV_BAD_WINDOW is set and the block's
 * rows see no key. */
typedef struct {
  int32_t num_blocks, block_len, max_pages, reserved;
  const int32_t *block_table;  /* [num_blocks, max_pages]                      */
  const int32_t *kv_len;       /* [num_blocks]                                 */
  const int32_t *window;       /* [num_blocks]; NULL = every block full        */
  const uint8_t *q_visible;    /* [num_blocks * block_len]; NULL = all visible */
  int32_t *vis_stats;          /* optional output [num_blocks*block_len, 3]:
                                  visible-key count, first and last visible
                                  key (-1 when none), as the kernel's own mask
                                  applied them; NULL = not written            */
} mla_attn_desc_t;

/* Blocks that share a context (MLA blog, forward_impl: the prefill path,
 * forward_mha with _compute_prefill_context, runs the expanded form when
 * many query rows meet one cached context).  Context c's blocks are
 * ctx_block_start[c] .. ctx_block_start[c+1]-1 (consecutive; the whole list
 * covers blocks 0 .. num_blocks-1).  Each block b of context c sees keys
 * 0 .. ctx_len[c]-1 as the context -- the same cache entries for all of c's
 * blocks, read through the table of block ctx_block_start[c] -- and keys
 * ctx_len[c] .. kv_len[b]-1 as its own, at most block_len of them
 * (kv_len[b] <= ctx_len[c] + block_len; a longer kv_len is reported on the
 * device as MLA_DEV_BAD_LENGTH and its extra keys are not seen).  The
 * visibility rule of mla_attn_desc_t applies unchanged. */
typedef struct {
  int32_t num_ctx;                 /* contexts, 1 .. num_blocks (else
                                      MLA_ERR_INVALID_ARG)                       */
  int32_t ctx_rows;                /* host: sum of ctx_len (keys of all contexts) */
  const int32_t *ctx_len;          /* device [num_ctx]                           */
  const int32_t *ctx_block_start;  /* device [num_ctx + 1]                       */
} mla_shared_ctx_t;

typedef struct mla_handle mla_handle_t;

/* ---- geometry (host only; no GPU needed) --------------------------------
 * MLA blog, MLAAttention.__init__ / get_kv_cache_shape: one cache entry is
 * kv_lora_rank + qk_rope_head_dim wide (576 for DeepSeek dims), one KV head;
 * MLAAttentionSpec.real_page_size_bytes: page bytes = page_size * 1 *
 * entry * dtype size.  Return 0 for a NULL or inconsistent config. */
int32_t mla_cache_entry_dim(const mla_config_t *cfg);
size_t mla_cache_page_bytes(const mla_config_t *cfg);

/* Bytes of the derived-weight arena mla_draft_init fills (0 = invalid cfg). */
size_t mla_weight_arena_bytes(const mla_config_t *cfg);

/* Validate `cfg` (returns MLA_ERR_INVALID_ARG / MLA_ERR_UNSUPPORTED with a
 * message), re-lay the weights out into the caller's device `arena`
 * (>= mla_weight_arena_bytes): W_UK / W_UV split out of kv_b_proj (MLA blog,
 * forward_impl: W_UK_T and _v_up_proj), the A-projection rows ordered
 * [kv | q | gate], a RoPE cos/sin table computed in fp64 on the host, and the
 * device status word.  Synchronises `stream` before returning; `w` is not
 * retained.  On success *out receives a handle owned by the caller (free with
 * mla_draft_destroy).  One handle serves one stream at a time. */
mla_status_t mla_draft_init(const mla_config_t *cfg, const mla_weights_t *w,
                            void *arena, size_t arena_bytes, void *stream,
                            mla_handle_t **out);

/* Device scratch needed by one append of n tokens / one forward of
 * num_tokens block tokens. */
size_t mla_append_workspace_bytes(const mla_handle_t *h, int32_t n);
size_t mla_forward_workspace_bytes(const mla_handle_t *h, int32_t num_tokens);

/* Latent-cache append (target-context injection, PR #758; MLA blog,
 * do_kv_cache_update): for each of the n tokens,
 *   kv = hidden[t] @ W_kva^T            (W_kva = last kv_lora_rank+qk_rope rows
 *                                         of fused_qkv_a_proj, or
 *                                         kv_a_proj_with_mqa)
 *   cache[slot_mapping[t]] = [RMSNorm(kv[:r]) * kv_a_layernorm |
 *                             RoPE(kv[r:], positions[t])]
 * hidden: device [n, hidden_size]; positions: device int32 [n];
 * slot_mapping: device int64 [n], slot = page * page_size + row;
 * cache: device [num_pages, page_size, entry].  n == 0 is a no-op. */
mla_status_t mla_latent_cache_append(mla_handle_t *h, const void *hidden,
                                     const int32_t *positions,
                                     const int64_t *slot_mapping, int32_t n,
                                     void *cache, int32_t num_pages,
                                     void *workspace, size_t workspace_bytes,
                                     void *stream);

/* Draft-layer forward for desc->num_blocks blocks of desc->block_len tokens
 * (MLA blog, wrapper forward + forward_impl MQA branch; PR #758 masks, gate):
 *   q = rope(q_b_proj(RMSNorm(q_c)))  (or q_proj), absorbed with W_UK;
 *   latent attention over the cache keys each block sees (mla_attn_desc_t);
 *   o = W_UV * latent output, optionally * sigmoid(hidden @ gate_proj^T);
 *   out = o @ o_proj^T.
 * hidden: device [nb*T, hidden_size]; positions: device int32 [nb*T];
 * block_slot_mapping: device int64 [nb*T] -- when non-NULL the block's own
 * latents are written to the cache there before attending; when NULL they
 * must already be in the cache (mla_latent_cache_append).  out: device
 * [nb*T, hidden_size].  Fully masked query rows come out as exact +0.
 * Any block_len.  bf16 layers run the tensor-core kernels, which need
 * kv_lora_rank 512, qk_rope_head_dim 64, a page_size of 16, 32, 64 or a
 * multiple of 128, hidden_size, q_lora_rank, qk_nope_head_dim and
 * num_heads * v_head_dim multiples of 64; mla_draft_init rejects other bf16
 * shapes with MLA_ERR_UNSUPPORTED (the fp32 layer has no such limits).  The
 * workspace must be 256-byte aligned. */
mla_status_t mla_draft_forward(mla_handle_t *h, const void *hidden,
                               const int32_t *positions,
                               const int64_t *block_slot_mapping, void *cache,
                               int32_t num_pages, const mla_attn_desc_t *desc,
                               void *out, void *workspace,
                               size_t workspace_bytes, void *stream);

/* mla_draft_forward whose attention waits for an event.  Everything that
 * does not read the cache -- the projections, query RoPE and W_UK
 * absorption, and the block's own latents when block_slot_mapping is
 * non-NULL -- is enqueued on `stream` at once; before the attention, the
 * stream waits for `cache_ready` (a cudaEvent_t the caller recorded after
 * the cache writes the attention reads, typically mla_latent_cache_append
 * of the target context on another stream).  The block's projections then
 * run while the context is appended (the pages' draft reads the context
 * only through the attention's keys).  The two must write disjoint slots;
 * an append that needs a workspace needs its own.  cache_ready == NULL is
 * exactly mla_draft_forward.  Graph-capturable: recorded into a stream
 * capture, the event forks and joins the two streams.  Same arguments,
 * results and errors as mla_draft_forward otherwise. */
mla_status_t mla_draft_forward_after(mla_handle_t *h, const void *hidden,
                                     const int32_t *positions,
                                     const int64_t *block_slot_mapping, void *cache,
                                     int32_t num_pages, const mla_attn_desc_t *desc,
                                     void *out, void *workspace,
                                     size_t workspace_bytes, void *stream,
                                     void *cache_ready);

/* mla_draft_forward for blocks that share contexts (mla_shared_ctx_t), in
 * the expanded form when the layer allows it (bf16, kv_lora_rank 512,
 * qk_rope_head_dim 64, qk_nope_head_dim and v_head_dim 128, block_len <=
 * 128): each context's latents and each block's
 * own latents are expanded once by kv_b_proj into per-head k_nope and v
 * (MLA blog, forward_mha: kv_b_proj on the prefill context), the queries
 * keep q_nope and q_pe (no W_UK / W_UV absorption), and one attention runs
 * per (head, up to 128 / block_len blocks of a context): the context keys,
 * then the blocks' own keys as one more key tile, masked to each block's
 * own.  Other layers run mla_draft_forward.  Same results and errors as
 * mla_draft_forward, plus MLA_ERR_INVALID_ARG for a NULL context list or one
 * outside its contract (num_ctx not in 1 .. num_blocks, ctx_rows < 0); the
 * workspace (256-byte aligned, caller-owned) is
 * mla_forward_shared_workspace_bytes(h, num_tokens, ctx_rows) bytes, 0 for
 * a NULL handle or negative counts. */
size_t mla_forward_shared_workspace_bytes(const mla_handle_t *h, int32_t num_tokens,
                                          int32_t ctx_rows);
mla_status_t mla_draft_forward_shared(mla_handle_t *h, const void *hidden,
                                      const int32_t *positions,
                                      const int64_t *block_slot_mapping, void *cache,
                                      int32_t num_pages, const mla_attn_desc_t *desc,
                                      const mla_shared_ctx_t *ctx, void *out,
                                      void *workspace, size_t workspace_bytes,
                                      void *stream);

/* mla_draft_forward_shared whose attention waits for an event, as
 * mla_draft_forward_after: everything before the gather of the cache rows
 * is enqueued at once, then the stream waits for `cache_ready`. */
mla_status_t mla_draft_forward_shared_after(mla_handle_t *h, const void *hidden,
                                            const int32_t *positions,
                                            const int64_t *block_slot_mapping, void *cache,
                                            int32_t num_pages, const mla_attn_desc_t *desc,
                                            const mla_shared_ctx_t *ctx, void *out,
                                            void *workspace, size_t workspace_bytes,
                                            void *stream, void *cache_ready);

/* The attention step of mla_draft_forward_shared alone, on the intermediates
 * the last such call left in `workspace` (same handle, descriptor, context
 * list and token count): the queries' q_nope and q_pe, the gathered latent
 * rows and their kv_b_proj expansion, the gate.  It rewrites the workspace's
 * per-head output o (the input of o_proj) with the same values the forward
 * computed.  For timing and checking that step in isolation.
 * MLA_ERR_UNSUPPORTED when the layer does not take the expanded form,
 * MLA_ERR_INVALID_ARG for NULL pointers, a context list outside its contract
 * or a workspace smaller than mla_forward_shared_workspace_bytes(). */
mla_status_t mla_shared_attention(mla_handle_t *h, const int32_t *positions,
                                  const mla_attn_desc_t *desc, const mla_shared_ctx_t *ctx,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Allocation-free latent-cache append.  The pages have no counterpart: this
 * is a library convenience for callers that cannot allocate device memory
 * where they append (host callbacks, allocator hooks, runtimes with a memory
 * pool fixed in advance, embedders that only hand over tensors they own).
 * Same result as mla_latent_cache_append, same arguments minus the
 * workspace: the fp32 staging of the projection lives in a fixed 4 MiB
 * device array inside the library, held by every GPU that loads it until
 * the process exits.  Limits and rules:
 *  - n * (kv_lora_rank + qk_rope_head_dim) must fit 2^20 floats
 *    (mla_append_noalloc_max_tokens(h) tokens, 1820 at entry width 576);
 *    larger n returns MLA_ERR_INVALID_ARG with a message, nothing launched;
 *  - the handle's device must be current; the first call on each device
 *    looks up the array's device address (cudaGetSymbolAddress), so make
 *    that first call before any stream capture; the address is kept for the
 *    life of the process, so this entry point must not be used after the
 *    device has been reset (cudaDeviceReset destroys the array);
 *  - every call shares the one array per device: calls whose work overlaps
 *    on the GPU (other streams, other handles, other threads) race on it and
 *    must be ordered by the caller.  Nothing in it needs to start at zero.
 * Calls no cudaMalloc/cudaFree and no allocating library routine. */
mla_status_t mla_latent_cache_append_noalloc(mla_handle_t *h, const void *hidden,
                                             const int32_t *positions,
                                             const int64_t *slot_mapping, int32_t n,
                                             void *cache, int32_t num_pages, void *stream);
int64_t mla_append_noalloc_max_tokens(const mla_handle_t *h);

/* Byte offset inside a forward workspace (sized for num_tokens block tokens)
 * of an intermediate the forward leaves there: MLA_WS_Q_ABS, the absorbed
 * queries [num_tokens, H, kv_lora_rank + qk_rope_head_dim] in the cache dtype,
 * MLA_WS_O_LAT, the latent attention output [num_tokens, H, kv_lora_rank]
 * (fp16 for bf16 layers, fp32 for fp32 layers), or MLA_WS_O, the per-head
 * output [num_tokens, H, v_head_dim] that o_proj reads (same types; in a
 * workspace of mla_draft_forward_shared too, at the same offsets); in a
 * workspace of mla_draft_forward_tree only (the others end there), MLA_WS_LSE,
 * the log-sum-exp of its attention's rows, fp32 [num_tokens, H].  Valid after the forward's
 * work on the stream has completed, until the workspace is reused.  Returns
 * (size_t)-1 for a NULL handle, a negative count or an unknown part. */
size_t mla_forward_workspace_offset(const mla_handle_t *h, int32_t num_tokens,
                                    int32_t part);

/* The latent attention step alone (MLA blog, forward_mqa and the Triton
 * decode_attention_fwd it calls, which returns the output and the
 * log-sum-exp of each query row; PR #758 / PR #1026 masks and zeroing):
 * for every row m = (token, head) of q_abs,
 *   s_j = scale * <q_abs[m], cache entry of key j>   over the visible keys j
 *   o_lat[m] = sum_j softmax(s)_j * entry_j[:kv_lora_rank]
 *   lse[m]   = log sum_j exp(s_j)                     (natural log)
 * with visibility and the key -> cache-slot walk of mla_attn_desc_t.  A row
 * that sees no key gets o_lat = +0 exactly and lse = -inf.
 * q_abs: device [nb*T, H, kv_lora_rank + qk_rope_head_dim] in the cache dtype
 * (bf16 or fp32), 16-byte aligned; positions: device int32 [nb*T]; cache as
 * for the forward; o_lat: device [nb*T, H, kv_lora_rank], fp16 for bf16
 * layers (the forward's intermediate type), fp32 for fp32 layers; lse:
 * device fp32 [nb*T, H] or NULL.  The cache is only read.  Blocks of at
 * most 32 query rows (block_len * num_heads <= 32, bf16, page_size a
 * multiple of 128) run a kernel for few rows that splits every block's keys
 * across the SMs and merges the splits by log-sum-exp (the blog's
 * forward_mqa num_kv_splits / merge_attn_states); it needs a device
 * workspace of mla_latent_attention_workspace_bytes() (256-byte aligned;
 * MLA_ERR_INVALID_ARG when smaller), other shapes need none (workspace may be
 * NULL).  Asynchronous on `stream`; no allocation.  Index errors are
 * reported through the device status word like the forward's. */
size_t mla_latent_attention_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc);
mla_status_t mla_latent_attention(mla_handle_t *h, const void *q_abs,
                                  const int32_t *positions, const void *cache,
                                  int32_t num_pages, const mla_attn_desc_t *desc,
                                  void *o_lat, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Backward of the latent attention step (the draft layer is trained through
 * it: "Add config-selectable MLA draft attention" (SpecForge PR #758),
 * Validation, gradient parity; forward = mla_latent_attention).  With
 * P = exp(scale * <q_abs[i], e_j> - lse[i]) over the visible keys j of row
 * i, dP = d_o_lat[i] . e_j[:kv_lora_rank], D = d_o_lat[i] . o_lat[i] and
 * dS = P (dP - D):
 *   d_q_abs[i] = scale * sum_j dS_ij e_j                        (written)
 *   d_cache[slot(j)] += scale * sum_i dS_ij q_abs[i]
 *                       + sum_i P_ij d_o_lat[i] on its first kv_lora_rank
 *                         columns (the entries are keys and values at once)
 * over every block of `desc` (blocks whose keys share cache pages add into
 * the same slots; the caller zeroes d_cache before the first call).  Rows
 * without a visible key pass nothing back.  q_abs, positions, cache, desc as
 * for mla_latent_attention; o_lat and lse are that call's outputs; d_o_lat,
 * d_q_abs: device fp32 [nb*T, H, ...]; d_cache: device fp32 [num_pages *
 * page_size, kv_lora_rank + qk_rope_head_dim].  SIMT kernels, fp32
 * arithmetic; entries at most 640 wide (MLA_ERR_UNSUPPORTED otherwise).
 * Asynchronous on `stream`; no allocation. */
mla_status_t mla_latent_attention_backward(mla_handle_t *h, const void *q_abs,
                                           const int32_t *positions, const void *cache,
                                           int32_t num_pages, const mla_attn_desc_t *desc,
                                           const void *o_lat, const float *lse,
                                           const float *d_o_lat, float *d_q_abs,
                                           float *d_cache, void *stream);

/* ---- trees of drafted tokens, and a cache of bounded length --------------
 * One verification step of speculative decoding over the latent cache: the
 * drafted tree attends the cache, the weight that every cached key received
 * is accumulated, and from time to time the keys with little weight leave the
 * cache.  The accepted path of a tree is kept by the same compaction.
 *
 * A block of T = block_len nodes is the tail of its sequence: logical keys
 * 0 .. kv_len - T - 1 are the context and key kv_len - T + k is node k's own.
 * parent: device int32 [num_blocks * block_len], per block: -1 for a child of
 * the context, else the index of an earlier node of the block (parent < node).
 * A node whose parent is below -1 (padding), and every node under it, is not
 * in the tree: its row sees no key and no row sees its key, whose entry and
 * position may hold anything.  A parent >= the node is reported as MLA_DEV_BAD_TREE and
 * treated the same.  Node i sees, with q_visible and window as in
 * mla_attn_desc_t, the context keys j with window == 0 or positions[i] - j <
 * window, and of the own keys those of the nodes a on its path from the
 * context, itself included, with window == 0 or positions[i] - positions[a] <
 * window.  positions are token positions: siblings share one.  A kv_len below
 * T or behind the page table is reported as MLA_DEV_BAD_LENGTH and the block's
 * rows see no key.  A chain (parent[i] = i - 1) is causal attention inside the
 * block; T = 1 is the one-token decode.  At most 1024 nodes a block
 * (MLA_ERR_UNSUPPORTED beyond).  Entries of the context that a window leaves
 * to some rows only, and of the tree's nodes, must be finite; entries that no
 * row sees may hold anything; a NaN that every row sees makes o_lat and lse
 * NaN. */

/* Latent attention of trees: mla_latent_attention with the visibility above
 * (same q_abs, cache, desc, o_lat, lse; vis_stats counts what a node sees).
 *   s_j = scale * <q_abs[m], entry_j>,  o_lat = sum_j softmax(s)_j entry_j[:r],
 *   lse = log sum_j exp(s_j)
 * workspace: mla_tree_attention_workspace_bytes() bytes, 256-byte aligned
 * (NULL when that is 0).  The launch and its workspace are planned from
 * max_pages and from whether window is NULL, since lengths and windows are on
 * the device: a table much wider than its sequences, and windows that leave
 * long ranges (0 among them), are right but slower. */
size_t mla_tree_attention_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc);
mla_status_t mla_tree_attention(mla_handle_t *h, const void *q_abs, const int32_t *positions,
                                const void *cache, int32_t num_pages,
                                const mla_attn_desc_t *desc, const int32_t *parent,
                                void *o_lat, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream);

/* The whole layer over trees: mla_draft_forward with the tree's visibility in
 * its attention (same arguments, results and errors; block_slot_mapping
 * writes the nodes' own entries first; padding nodes take a free slot of
 * their own and a position inside the table).  cache must be 16-byte aligned,
 * on fp32 layers too.  The workspace keeps the absorbed queries and their
 * log-sum-exps (mla_forward_workspace_offset, MLA_WS_Q_ABS and MLA_WS_LSE),
 * from which mla_key_weights goes on. */
size_t mla_forward_tree_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc);
mla_status_t mla_draft_forward_tree(mla_handle_t *h, const void *hidden,
                                    const int32_t *positions,
                                    const int64_t *block_slot_mapping, void *cache,
                                    int32_t num_pages, const mla_attn_desc_t *desc,
                                    const int32_t *parent, void *out, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* The attention weight that every key of a block received from the block's
 * rows, added to what it had:
 *   weights_out[b, j] = decay * prior[b, j] + sum_m exp(scale <q_abs[m], entry_j> - lse[m])
 * over the rows m = (query, head) of block b that see key j, for j < kv_len[b]
 * (other elements are left as they are).  parent: the tree's (NULL: the rule
 * of mla_attn_desc_t).  lse: device fp32 [nb*T, H], mla_tree_attention's or
 * mla_latent_attention's for the same rows; a row with lse = -inf (so those
 * that see no key, nodes outside the tree among them) adds nothing.  prior,
 * weights_out: device fp32 [num_blocks, ldw], the same pointer or disjoint;
 * prior may be NULL (nothing before).  ldw < kv_len is reported as
 * MLA_DEV_BAD_LENGTH and the keys behind it are left out.  Each
 * key's sum is taken in one fixed order: equal calls give equal bits.
 * vis_stats of desc is not written.  q_abs and cache 16-byte aligned.
 * workspace: mla_key_weights_workspace_bytes() bytes, 256-byte aligned (NULL
 * when that is 0). */
size_t mla_key_weights_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc,
                                       int64_t ldw);
mla_status_t mla_key_weights(mla_handle_t *h, const void *q_abs, const int32_t *positions,
                             const void *cache, int32_t num_pages, const mla_attn_desc_t *desc,
                             const int32_t *parent, const float *lse, float decay,
                             const float *prior, float *weights_out, int64_t ldw,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Which keys of a sequence stay when it may hold `budget` of them: all when
 * kv_len <= budget, else the first `sink`, the last `recent` and, of the
 * others, the budget - sink - recent with the largest weights (equal weights:
 * the lower index; NaN counts as less than -inf).  weights: device fp32
 * [num_seqs, ldw]; keep: device int32 [num_seqs, budget], ascending indices,
 * -1 behind the last; keep_len: device int32 [num_seqs].  kv_len > ldw is
 * reported as MLA_DEV_BAD_LENGTH and taken as ldw. */
mla_status_t mla_cache_select(mla_handle_t *h, const float *weights, int64_t ldw,
                              const int32_t *kv_len, int32_t num_seqs, int32_t budget,
                              int32_t sink, int32_t recent, int32_t *keep, int32_t *keep_len,
                              void *stream);

/* Moves the kept entries of every sequence together.  Row d of sequence b
 * becomes its row src(d): d for d < first[b], keep[b, d - first[b]] for the
 * keep_len[b] rows from first[b] on; keep (device int32 [num_seqs, ldk]) is
 * ascending, every index in [first[b], kv_len[b]).  first: device int32
 * [num_seqs], NULL = 0.  Eviction takes mla_cache_select's lists; an accepted
 * path takes first = context length and keep = the accepted nodes' keys.
 * The new length is first[b] + keep_len[b]; rows behind it are left as they
 * are.  Entries are moved as they are: their rotation stays that of their old
 * position, so positions go on counting tokens while logical indices move
 * up.  A sliding window counts logical indices of the context: after an
 * eviction use window 0.
 *   dst_block_table NULL: in place.  No page that holds a row from first[b] on
 * may belong to two sequences of the call (or twice to one); pages wholly
 * before first[b], a shared prompt's, are neither read nor written.  Else the rows go to the pages of
 * dst_block_table [num_seqs, dst_max_pages], none of which is read by the call
 * and none named twice.
 *   weights, weights_out: NULL, or device fp32 [num_seqs, ldw], moved the same
 * way (weights_out == weights exactly in place); elements first + keep_len ..
 * kv_len - 1 of weights_out become 0.
 * Reported on the device: a bad page (the row, its weight too, is left alone),
 * a kv_len beyond the table or ldw, and (MLA_DEV_BAD_KEEP) keep_len > ldk or >
 * kv_len - first (the sequence is left alone), and an index outside
 * its sequence or not above the one before it: in place the whole sequence is
 * left alone then, into other pages that row.
 * cache: 4-byte aligned (16-byte aligned is faster).
 * workspace: mla_cache_compact_workspace_bytes() bytes, 256-byte aligned,
 * needed in place only; two calls that may overlap on the GPU need two. */
size_t mla_cache_compact_workspace_bytes(const mla_handle_t *h, int32_t num_seqs, int64_t ldk);
mla_status_t mla_cache_compact(mla_handle_t *h, void *cache, int32_t num_pages,
                               const int32_t *block_table, int32_t max_pages,
                               const int32_t *kv_len, int32_t num_seqs, const int32_t *keep,
                               int64_t ldk, const int32_t *keep_len, const int32_t *first,
                               const int32_t *dst_block_table, int32_t dst_max_pages,
                               const float *weights, float *weights_out, int64_t ldw,
                               void *workspace, size_t workspace_bytes, void *stream);

/* ---- the latent cache in 8 bits ------------------------------------------
 * bf16 layers.  An entry of 576 bf16 numbers (1152 bytes) is kept in 644: its
 * 512 latent dims in e4m3 over one power of two of its own, its 64 rotary dims
 * in bf16 as they are.  Three arrays, page by page like the bf16 cache:
 *   latent: device e4m3 [num_pages, page_size, 512], 16-byte aligned
 *   rope:   device bf16 [num_pages, page_size, 64], 16-byte aligned
 *   scale:  device fp32 [num_pages, page_size], 16-byte aligned
 * and the entry stands for latent * scale and rope.  scale is the least power of two
 * that brings the latent's largest magnitude to 448 or below, 2^-64 at least; the
 * elements are rounded to nearest, ties to even (off by 2^-4 of their value at
 * most, or 2^-10 scale below 2^-6 scale).  Reading back into bf16 is exact, and what
 * was read back and is stored again stands for the same numbers.  An entry with an
 * element that is NaN, infinite, or a latent of 2^127 or more has scale NaN and
 * latent 0: its latent reads back as NaN, a row that sees it becomes NaN, and
 * rows that do not see it are as without it.
 *   The attention takes a scale by its exponent: of entries written by other means, too,
 * every scale that a row sees must be a power of two, 2^-64 .. 2^119 (or NaN).  Another
 * number is reported as MLA_DEV_BAD_SCALE and counts as NaN.  (mla_cache8_load multiplies by whatever
 * number it finds and rounds to bf16.) */
typedef struct {
  void *latent, *rope;
  float *scale;
} mla_cache8_t;

/* Entries into the 8-bit cache: entry t (device bf16 [n, 576], 16-byte aligned)
 * goes to slot slot_mapping[t] (device int64 [n], slot = page * page_size + row).
 * A slot outside the cache is reported as MLA_DEV_BAD_SLOT and skipped; of a slot
 * named twice one entry stays, or parts of both.  n == 0 is a no-op. */
mla_status_t mla_cache8_store(mla_handle_t *h, const void *entries, const int64_t *slot_mapping,
                              int32_t n, const mla_cache8_t *cache, int32_t num_pages, void *stream);

/* Entries read back: row t of entries (device bf16 [n, 576], 16-byte aligned)
 * becomes the entry of slot slot_mapping[t].  A slot outside the cache is reported
 * as MLA_DEV_BAD_SLOT and its row left as it is. */
mla_status_t mla_cache8_load(mla_handle_t *h, const mla_cache8_t *cache, int32_t num_pages,
                             const int64_t *slot_mapping, int32_t n, void *entries, void *stream);

/* mla_latent_cache_append into the 8-bit cache: the entries are rounded to bf16 as
 * the bf16 cache would hold them and stored as mla_cache8_store does.
 * workspace: mla_append8_workspace_bytes() bytes, 256-byte aligned. */
size_t mla_append8_workspace_bytes(const mla_handle_t *h, int32_t n);
mla_status_t mla_latent_cache_append8(mla_handle_t *h, const void *hidden,
                                      const int32_t *positions, const int64_t *slot_mapping,
                                      int32_t n, const mla_cache8_t *cache, int32_t num_pages,
                                      void *workspace, size_t workspace_bytes, void *stream);

/* Latent attention over the 8-bit cache: mla_latent_attention (parent NULL) or
 * mla_tree_attention (parent as there, at most 1024 nodes a block) with the
 * entries that the cache stands for; same q_abs, positions, desc, o_lat, lse,
 * same checks on the device, any block_len.  Entries that no row sees may hold
 * anything.  num_pages * page_size < 2^31.  Every block's keys are split over the SMs and joined by
 * log-sum-exp.
 *   Rounding: a softmax weight is held to 2^-8 of itself, and weight times scale to 2^-20 of the row's
 * largest such product; a query's elements exactly down to 2^-10 of the row's largest, and to 2^-17 of it
 * below; scores, sums and log-sum-exps in fp32; o_lat in fp16.  (Outputs are half as far from the exact ones
 * as those of mla_latent_attention and mla_tree_attention over the same entries in bf16.)  A key whose weight times
 * scale is below 2^-120 of the row's largest adds nothing to the sums; zeros have scale 2^-64.
 *   workspace: mla_latent_attention8_workspace_bytes() bytes,
 * 256-byte aligned; two calls that may overlap on the GPU need two. */
size_t mla_latent_attention8_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc);
mla_status_t mla_latent_attention8(mla_handle_t *h, const void *q_abs, const int32_t *positions,
                                   const mla_cache8_t *cache, int32_t num_pages,
                                   const mla_attn_desc_t *desc, const int32_t *parent,
                                   void *o_lat, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* The whole layer over the 8-bit cache: mla_draft_forward (parent NULL) or
 * mla_draft_forward_tree with mla_latent_attention8 as its attention and the block's own
 * entries written as mla_latent_cache_append8 writes them.  workspace:
 * mla_forward8_workspace_bytes() bytes, 256-byte aligned, with mla_draft_forward's
 * intermediates (mla_forward_workspace_offset, not MLA_WS_LSE). */
size_t mla_forward8_workspace_bytes(const mla_handle_t *h, const mla_attn_desc_t *desc);
mla_status_t mla_draft_forward8(mla_handle_t *h, const void *hidden, const int32_t *positions,
                                const int64_t *block_slot_mapping, const mla_cache8_t *cache,
                                int32_t num_pages, const mla_attn_desc_t *desc,
                                const int32_t *parent, void *out, void *workspace,
                                size_t workspace_bytes, void *stream);

/* mla_cache_compact of an 8-bit cache: the same arguments, results and checks on the device
 * (entries move with their scales).  workspace: mla_cache8_compact_workspace_bytes() bytes,
 * 256-byte aligned, needed in place only. */
size_t mla_cache8_compact_workspace_bytes(const mla_handle_t *h, int32_t num_seqs, int64_t ldk);
mla_status_t mla_cache8_compact(mla_handle_t *h, const mla_cache8_t *cache, int32_t num_pages,
                                const int32_t *block_table, int32_t max_pages,
                                const int32_t *kv_len, int32_t num_seqs, const int32_t *keep,
                                int64_t ldk, const int32_t *keep_len, const int32_t *first,
                                const int32_t *dst_block_table, int32_t dst_max_pages,
                                const float *weights, float *weights_out, int64_t ldw,
                                void *workspace, size_t workspace_bytes, void *stream);

/* ---- verification of drafted tokens ---------------------------------------
 * Which of a sequence's num_nodes drafted tokens (T) the target keeps, and the
 * token behind them, from given random numbers, so that what is kept is
 * distributed as the target's own tokens.  Node i drafts tokens[b, i] after its
 * parent (device int32 [num_seqs, T]; -1: after the context; -2: not in the tree; NULL:
 * the chain parent[i] = i - 1).  target [num_seqs, T + 1, ldt]: row 0 the
 * target's probabilities after the context, row i + 1 those after node i; draft
 * [num_seqs, T, ldd]: row 0 the distribution from which the context's children
 * were drawn, each for itself, row i + 1 that of node i's children; NULL: every token was
 * certain (a likeliest one, siblings distinct).  Both of `dtype` (MLA_FP32,
 * MLA_BF16, MLA_FP16), the first `vocab` elements of each row; an element that is
 * negative, NaN or infinite counts as 0.
 *   The sequence stands at the context (w = target row 0, s = 1).  Its nodes are
 * looked at in their order; one whose parent is where the sequence stands is taken if
 *   uniforms[b, i] s q(x) < w(x)       (x = tokens[b, i], q the draft's row there, 1 for NULL)
 * and the sequence then stands at it (w = target row i + 1, s = 1); else w becomes
 * max(w - s q, 0) and s its sum (draft NULL: w(x) becomes 0 and s loses it).
 * At the end next_token[b] is the least x with sum_{y <= x} w(y) >
 * uniforms[b, T] sum w.  Where nothing is left of w it is drawn from the target's row
 * itself; without any mass there it is -1 (MLA_DEV_BAD_DRAFT).
 *   accepted: device int32 [num_seqs, T], the taken nodes in order, first[b] added
 * to each (device int32 [num_seqs], NULL = 0), -1 behind the last; num_accepted: device
 * int32 [num_seqs].  With first = context length they are mla_cache_compact's
 * keep, keep_len and first.  uniforms: device fp32 [num_seqs, T + 1] in [0, 1).
 * A token outside the vocabulary is reported as MLA_DEV_BAD_DRAFT, its node
 * refused and w left as it was; a parent >= the node as MLA_DEV_BAD_TREE, its
 * node never reached.  Sums and differences are carried to 2^-40 or better.  T at most
 * 1024 (MLA_ERR_UNSUPPORTED beyond); T == 0 draws from row 0. */
mla_status_t mla_verify_drafts(mla_handle_t *h, const void *target, int64_t ldt, const void *draft,
                               int64_t ldd, int32_t dtype, const int32_t *tokens,
                               const int32_t *parent, const float *uniforms, const int32_t *first,
                               int32_t num_seqs, int32_t num_nodes, int32_t vocab,
                               int32_t *accepted, int32_t *num_accepted, int32_t *next_token,
                               void *stream);

/* Synchronise `stream`, read and clear the device status word.  Returns
 * MLA_OK, MLA_ERR_TIMEOUT (MLA_DEV_TIMEOUT set) or MLA_ERR_DEVICE_CHECK; the
 * raw bits go to *bits when non-NULL. */
mla_status_t mla_get_device_status(mla_handle_t *h, void *stream, int32_t *bits);

/* Self-check of the failure path (no counterpart on the pages: a test aid
 * for the bounded waits every kernel of the library uses).  Enqueues one
 * single-thread kernel that waits, with the library's bounded mbarrier wait,
 * on a barrier nothing ever arrives on; after max_rounds try_wait rounds
 * (1 .. 2^24; the kernels themselves use 2^26) the wait gives up, sets
 * MLA_DEV_TIMEOUT in the handle's device status word and writes 1 to
 * *gave_up (device int32).  The kernel issues no copies and holds no tensor
 * memory, so nothing is in flight when it returns and the handle stays
 * usable: mla_get_device_status then returns MLA_ERR_TIMEOUT once and clears
 * the word.  Asynchronous on `stream`. */
mla_status_t mla_check_wait_timeout(mla_handle_t *h, uint32_t max_rounds,
                                    int32_t *gave_up, void *stream);

/* Number of CUDA kernels this handle has enqueued so far (host counter;
 * launches replayed from a captured CUDA graph are not counted). */
unsigned long long mla_kernel_launches(const mla_handle_t *h);

void mla_draft_destroy(mla_handle_t *h);
const char *mla_status_string(mla_status_t s);
/* Message of the last failing call on this thread ("" if none). */
const char *mla_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MLA_DRAFT_H */
