/*
 * pe.h — C ABI of libpe.so: P-EAGLE parallel drafting and greedy
 * verify / batch-metadata rebuild on one GB300 (sm_103a).
 *
 * The method (cited by page title and section):
 *  - "在 Amazon SageMaker AI 上使用 P-EAGLE 并行化推测解码" (Chinese translation
 *    of the AWS post), section "解决方案概述" (Solution overview):
 *    "P-EAGLE 如何打破这个链" — learned placeholders emb_mask and h_shared;
 *    "逐步草稿过程" — Step 1: target hidden states of layers 2, L/2, L-1
 *    concatenated to 3d; Step 2: position 1 = real token embedding + target
 *    hidden, positions 2..K = emb_mask + h_shared, all K positions through
 *    the 4 drafter layers and the LM head in one pass, K drafts at once; the
 *    target then verifies all K in one pass with the standard acceptance rule.
 *  - "Amazon SageMaker AIにおけるP-EAGLEによる推論高速化": a fused kernel
 *    rebuilds the batch metadata after verification.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller unless stated
 *    otherwise; the library never frees them. Matrices are row-major,
 *    weight matrices are stored [out, in].
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Calls are
 *    asynchronous on that stream; outputs are valid once it reaches them.
 *  - The return value is PE_OK or a negative PE_ERR_* code; on error
 *    pe_last_error() (thread-local) describes it and nothing was enqueued.
 *  - Problems found on the device for one request (bad page index, cache
 *    capacity) are reported per request in `status[b]` (PE_REQ_*); other
 *    requests are unaffected. No kernel traps; every device-side wait is
 *    bounded and a wait that gives up sets a flag read by pe_device_errors().
 */
#ifndef PE_H
#define PE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PE_ABI_VERSION 1

/* return codes */
#define PE_OK               0
#define PE_ERR_ARG         -1   /* null pointer, size out of range, misaligned pointer */
#define PE_ERR_UNSUPPORTED -2   /* shape the kernels do not implement */
#define PE_ERR_CUDA        -3   /* a CUDA runtime / driver call failed */
#define PE_ERR_NOMEM       -4   /* workspace allocation failed */

/* per-request status written by pe_draft and pe_verify_rebuild */
#define PE_REQ_OK          0
#define PE_REQ_CAPACITY    1    /* entries needed exceed max_pages * page_size */
#define PE_REQ_BAD_PAGE    2    /* a needed page-table entry is outside [0, num_pages) */
#define PE_REQ_BAD_INPUT   3    /* token id outside [0, V), negative length */
#define PE_REQ_TIMEOUT     4    /* pe_attention_kv8, pe_attention_kv4: a device-side wait gave up; all outputs of the call are zero */

/* bits of the device error word (pe_device_errors) */
#define PE_DEVERR_GEMM_TIMEOUT  1u
#define PE_DEVERR_ATTN_TIMEOUT  2u
#define PE_DEVERR_CHAIN_TIMEOUT 4u   /* the persistent layer-chain kernel */

#define PE_DTYPE_BF16 0         /* bf16 weights/activations/KV, fp32 accumulate */
#define PE_DTYPE_FP32 1         /* fp32 everything; GEMMs run as tf32 */
#define PE_DTYPE_FP8W 2         /* FP8 (E4M3) GEMM weights with one fp32 scale per output row;
                                   bf16 activations, embeddings, norm gains and KV cache
                                   (pe_init_drafter_fp8) */

/* Drafter shape. n_layers must be 4, page_size 16, head_dim 64 or 128,
 * n_kv_heads must divide n_q_heads, n_q_heads*head_dim and
 * n_kv_heads*head_dim must be multiples of 128, hidden and ffn multiples
 * of 64. k_max (1..16) is the largest K any call will pass. */
typedef struct pe_config {
    int32_t hidden;       /* H */
    int32_t n_layers;     /* 4 */
    int32_t n_q_heads;    /* nq */
    int32_t n_kv_heads;   /* nkv */
    int32_t head_dim;     /* hd */
    int32_t ffn;          /* F (SwiGLU width) */
    int32_t vocab;        /* V */
    float   rms_eps;      /* RMSNorm epsilon */
    float   rope_theta;   /* RoPE base */
    int32_t page_size;    /* 16 */
    int32_t k_max;        /* largest K a call may pass */
    int32_t dtype;        /* PE_DTYPE_* for weights, activations and KV cache */
} pe_config;

/* Per-layer weights, all of the config dtype, device pointers, 16-byte aligned. */
typedef struct pe_layer_weights {
    const void* norm_e;     /* [H]  layer 0 only: gain of RMSNorm on the token embedding half */
    const void* norm_h;     /* [H]  layer 0 only: gain of RMSNorm on the hidden half */
    const void* attn_norm;  /* [H]  layers 1..3: pre-attention RMSNorm gain (NULL for layer 0) */
    const void* w_qkv;      /* [(nq+2nkv)*hd, in], in = 2H for layer 0, H otherwise; rows q | k | v */
    const void* w_o;        /* [H, nq*hd] */
    const void* mlp_norm;   /* [H]  pre-MLP RMSNorm gain */
    const void* w_gate;     /* [F, H] */
    const void* w_up;       /* [F, H] */
    const void* w_down;     /* [H, F] */
} pe_layer_weights;

typedef struct pe_weights {
    const void* fc;          /* [H, 3H]: fuses [h_lo; h_mid; h_hi] into H */
    const void* embed;       /* [V, H] token embedding */
    const void* emb_mask;    /* [H] learned mask-token embedding (positions 2..K) */
    const void* h_shared;    /* [H] learned shared hidden state (positions 2..K) */
    const void* final_norm;  /* [H] */
    const void* lm_head;     /* [V, H] (not tied to embed) */
    pe_layer_weights layer[4];
} pe_weights;

/* FP8 drafter weights. The pages run their benchmarks in FP8 ("在 Amazon
 * SageMaker AI 上使用 P-EAGLE 并行化推测解码", section "基准测试"); here every
 * GEMM weight matrix (FC, QKV, O, gate, up, down, LM head) may be given as
 * E4M3 codes q[m, k] (uint8, the same [out, in] layout, rows a multiple of 16
 * bytes) standing for W[m, k] = q[m, k] * scale[m]. The codes are widened to
 * bf16 in shared memory (exactly: every E4M3 value is a bf16 value), the
 * tensor cores multiply bf16 by bf16 with fp32 accumulation, and the epilogue
 * applies scale[m]. Each array below is fp32 [rows of that matrix]. Codes
 * must be finite: the NaN codes 0x7F / 0xFF are not decoded as NaN. */
typedef struct pe_layer_scales {
    const float* w_qkv;     /* [(nq+2nkv)*hd] */
    const float* w_o;       /* [H] */
    const float* w_gate;    /* [F] */
    const float* w_up;      /* [F] */
    const float* w_down;    /* [H] */
} pe_layer_scales;

typedef struct pe_weight_scales {
    const float* fc;        /* [H] */
    const float* lm_head;   /* [V] */
    pe_layer_scales layer[4];
} pe_weight_scales;

typedef struct pe_handle pe_handle;

/* Create a drafter on `device` (the device must be current or will be made
 * current). Records the weight pointers (caller keeps them alive until
 * pe_destroy), allocates the workspaces for up to max_batch requests of up to
 * cfg->k_max rows and builds TMA descriptors for the weights. Synchronous. */
int pe_init_drafter(const pe_config* cfg, const pe_weights* weights,
                    int32_t max_batch, int32_t device, pe_handle** out);

/* The same for FP8 weights: cfg->dtype must be PE_DTYPE_FP8W; the GEMM
 * matrices of `weights` point at E4M3 codes, the other entries (embed,
 * emb_mask, h_shared, norm gains) at bf16; `scales` gives the per-row scales
 * (device fp32, caller-owned like the weights). Every other entry point works
 * unchanged on the handle, with bf16 target hidden states and KV cache. The
 * persistent layer chain (PE_LAYER_CHAIN) is not used with FP8 weights. */
int pe_init_drafter_fp8(const pe_config* cfg, const pe_weights* weights, const pe_weight_scales* scales,
                        int32_t max_batch, int32_t device, pe_handle** out);

/* One parallel draft pass (pages' Step 2) for B requests, K drafts each.
 *
 *  last_token    [B] int32     last accepted token of each request (row 0 input)
 *  target_hidden [B, 3H]       config dtype; [h_lo | h_mid | h_hi] of that token
 *  positions     [B] int32     Q_b: RoPE position of row 0; row j uses Q_b + j
 *  seq_lens      [B] int32     S_b: committed drafter-cache entries; row j is
 *                              written to and attends through entry S_b + j
 *  page_table    [B, max_pages] int32  physical page of each 16-entry block
 *  num_pages     pages in each layer of the caches
 *  k_cache, v_cache  [4][num_pages][nkv][16][hd] config dtype; read for
 *                entries < S_b, written at entries S_b..S_b+K-1
 *  drafts        [B, K] int32  OUT: argmax of the LM head per row
 *  logits_dbg    [B, K, V] fp32 OUT or NULL: full logits (testing only)
 *  status        [B] int32     OUT: PE_REQ_*; a request that is not OK gets
 *                drafts -1 and no cache writes
 * Requires 1 <= B <= max_batch, 1 <= K <= k_max, target_hidden 16-byte aligned. */
int pe_draft(pe_handle* h, int32_t B, int32_t K,
             const int32_t* last_token, const void* target_hidden,
             const int32_t* positions, const int32_t* seq_lens,
             const int32_t* page_table, int32_t max_pages, int32_t num_pages,
             void* k_cache, void* v_cache,
             int32_t* drafts, float* logits_dbg, int32_t* status, void* stream);

/* Sequential (EAGLE-style) drafting on the same kernels: the chain that
 * P-EAGLE breaks ("在 Amazon SageMaker AI 上使用 P-EAGLE 并行化推测解码",
 * "P-EAGLE 如何打破这个链": each draft needs the embedding of the token drafted
 * just before it and the hidden state that produced it). K passes of one row
 * per request, each a full drafter forward:
 *  - pass 0 is the parallel pass's row 0 (embedding of last_token, FC-fused
 *    target hidden state);
 *  - pass j > 0 takes the embedding of draft j-1 and, as its hidden input and
 *    residual start, the drafter's own final residual stream of pass j-1
 *    (the hidden state before the final RMSNorm);
 *  - pass j sits at RoPE position Q_b + j and cache entry S_b + j and writes
 *    its k/v rows there before pass j+1 attends over them.
 * Same arguments, layouts, outputs and errors as pe_draft (drafts[b, j] is
 * pass j's argmax; logits_dbg row (b, j) its logits); every entry
 * S_b .. S_b+K-1 the step writes is validated by pass 0. The launch count
 * grows linearly in K (K forward passes), where pe_draft's does not. */
int pe_draft_sequential(pe_handle* h, int32_t B, int32_t K,
                        const int32_t* last_token, const void* target_hidden,
                        const int32_t* positions, const int32_t* seq_lens,
                        const int32_t* page_table, int32_t max_pages, int32_t num_pages,
                        void* k_cache, void* v_cache,
                        int32_t* drafts, float* logits_dbg, int32_t* status, void* stream);

/* The parallel draft pass with the tokens of the last verify re-fed as real
 * rows (the alternative to the single-real-row bookkeeping; the pages leave
 * the drafter's cache bookkeeping open). Request b brings n_b = n_real[b]
 * real rows - tokens[b, i] with their target hidden states target_hidden[b, i]
 * (each row: token embedding and FC-fused hidden state, the pages'
 * position-1 input) - ahead of the K-1 placeholder rows. Real row i sits at
 * position Q_b + i and entry S_b + i; placeholder j (1..K-1) at position
 * Q_b + n_b - 1 + j and entry S_b + n_b - 1 + j; every row attends causally.
 * drafts[b, 0] is the argmax of the last real row, drafts[b, j] that of
 * placeholder j.
 *  tokens        [B, n_max] int32 (entries past n_b unused), n_real [B] int32 in 1..n_max
 *  target_hidden [B, n_max, 3H] bf16 (rows past n_b unused)
 *  1 <= n_max <= k_max. Other arguments, outputs and errors as for pe_draft;
 *  every entry S_b .. S_b+n_max+K-2 is validated (PE_REQ_BAD_INPUT also for
 *  n_b out of range or a bad token).
 * Runs as two passes: the layers over real rows 0..n_b-2 (which writes their
 * cache rows; padded to n_max-1 rows, the padding writes nothing), then the
 * parallel pass whose row 0 is the last real row. The result is that of one
 * joint pass, because attention is the only place where rows meet. */
int pe_draft_refeed(pe_handle* h, int32_t B, int32_t K, int32_t n_max, const int32_t* tokens,
                    const int32_t* n_real, const void* target_hidden, const int32_t* positions,
                    const int32_t* seq_lens, const int32_t* page_table, int32_t max_pages, int32_t num_pages,
                    void* k_cache, void* v_cache, int32_t* drafts, float* logits_dbg, int32_t* status,
                    void* stream);

/* Greedy verification + batch-metadata rebuild + KV rollback (one kernel).
 * h may be NULL (the kernel needs no drafter state).
 *
 *  drafts        [B, K] int32     the step's drafts d
 *  target_tokens [B, K+1] int32   target argmax tokens g for the K+1 positions
 *  page_table    [B, max_pages] int32, num_pages as for pe_draft
 *  positions, seq_lens  [B] int32 in: Q_b, S_b of the step just drafted
 *  positions_out, seq_lens_out [B] int32 OUT (may alias the inputs):
 *                 Q_b' = Q_b + a_b + 1, S_b' = S_b + min(a_b, K-1) + 1
 *  accepted      [B] int32 OUT  a_b = longest prefix with d == g, 0..K
 *  bonus         [B] int32 OUT  g[b, a_b]
 *  emitted       [B, K+1] int32 OUT or NULL: d[b, :a_b], bonus, then -1
 *  slot_mapping  [B, K] int32 OUT  physical slot (page*16 + offset) of entries
 *                 S_b' .. S_b'+K-1 (where the next draft pass writes)
 *  rollback_slots [B, K] int32 OUT  slots of rejected entries S_b' .. S_b+K-1,
 *                 then -1 padding
 *  status        [B] int32 OUT  PE_REQ_*; when not OK, positions/seq_lens are
 *                 passed through unchanged and slot/rollback rows are -1.
 * Requires 1 <= K <= 31. */
int pe_verify_rebuild(pe_handle* h, int32_t B, int32_t K,
                      const int32_t* drafts, const int32_t* target_tokens,
                      const int32_t* page_table, int32_t max_pages, int32_t num_pages,
                      const int32_t* positions, const int32_t* seq_lens,
                      int32_t* positions_out, int32_t* seq_lens_out,
                      int32_t* accepted, int32_t* bonus, int32_t* emitted,
                      int32_t* slot_mapping, int32_t* rollback_slots,
                      int32_t* status, void* stream);

/* Verify + rebuild after a pe_draft_refeed pass: the same greedy acceptance,
 * bonus and emitted tokens; the n_b real rows stay committed and the K-1
 * placeholder rows are rolled back:
 *  n_real, positions, seq_lens [B] in; n_real_out = a_b + 1,
 *  positions_out = Q_b + n_b, seq_lens_out = S_b + n_b (may alias the inputs)
 *  slot_mapping  [B, 2K] OUT  slots of the next pass's entries
 *                 S_b' .. S_b'+n_b'+K-2, then -1
 *  rollback_slots [B, K] OUT  slots of entries S_b+n_b .. S_b+n_b+K-2, then -1
 *  status: as pe_verify_rebuild (PE_REQ_BAD_INPUT also for n_b outside
 *  1..K+1); a failed request keeps its metadata and n_real.
 * The next step re-feeds emitted[b, 0..a_b] with their target hidden states.
 * Requires 1 <= K <= 16. */
int pe_verify_rebuild_refeed(pe_handle* h, int32_t B, int32_t K, const int32_t* drafts,
                             const int32_t* target_tokens, const int32_t* page_table, int32_t max_pages,
                             int32_t num_pages, const int32_t* n_real, const int32_t* positions,
                             const int32_t* seq_lens, int32_t* n_real_out, int32_t* positions_out,
                             int32_t* seq_lens_out, int32_t* accepted, int32_t* bonus, int32_t* emitted,
                             int32_t* slot_mapping, int32_t* rollback_slots, int32_t* status, void* stream);

/* Sampled drafting and stochastic acceptance (the pages' "standard
 * acceptance criterion" when decoding samples, as their deployment does at
 * temperature 0.3: "在 Amazon SageMaker AI 上使用 P-EAGLE 并行化推测解码",
 * "逐步草稿过程"). With q_j = softmax(draft logits of row j / T) and
 * p_j = softmax(target logits of position j / T), speculative sampling
 * accepts draft d_j while u_j < p_j(d_j) / q_j(d_j), and emits at the first
 * rejection a token drawn from max(0, p_j - q_j) (normalised), or after K
 * acceptances a bonus token drawn from p_K; the emitted tokens are then
 * distributed as sampling the target alone. Every draw is inverse-CDF
 * sampling with a caller-supplied uniform u in [0, 1): the smallest index
 * whose running weight, summed in index order, exceeds u times the total.
 *
 * pe_sample_drafts: drafts[b, j] ~ q_j from logits [B, K, V] fp32 (the
 *  logits output of pe_draft / pe_draft_refeed; P-EAGLE's rows come from one
 *  pass, so each row is drawn independently), u [B, K] fp32; status [B]
 *  (nullable: requests not PE_REQ_OK get -1).
 * pe_verify_stochastic: draft_logits [B, K, V], target_logits [B, K+1, V]
 *  fp32, u_accept [B, K], u_final [B] fp32; accepted [B] OUT a_b,
 *  final_token [B] OUT the drawn token (it takes the place of the greedy
 *  bonus); emitted, the metadata rebuild, rollback and status exactly as
 *  pe_verify_rebuild given a_b. Uses the handle's workspace (h required;
 *  B <= max_batch, K <= k_max). temperature > 0. */
int pe_sample_drafts(pe_handle* h, int32_t B, int32_t K, const float* logits, float temperature, const float* u,
                     const int32_t* status, int32_t* drafts, void* stream);
int pe_verify_stochastic(pe_handle* h, int32_t B, int32_t K, const int32_t* drafts, const float* draft_logits,
                         const float* target_logits, float temperature, const float* u_accept, const float* u_final,
                         const int32_t* page_table, int32_t max_pages, int32_t num_pages, const int32_t* positions,
                         const int32_t* seq_lens, int32_t* positions_out, int32_t* seq_lens_out, int32_t* accepted,
                         int32_t* final_token, int32_t* emitted, int32_t* slot_mapping, int32_t* rollback_slots,
                         int32_t* status, void* stream);

/* The draft pass's tcgen05 GEMM engine on its own (plain store epilogue):
 *   y[n, m] = sum_k w[m, k] * x[n, k]
 *  w  [M, Kd] config-dtype weights, x [N, Kd] activations (same dtype),
 *  y  [N, M] fp32 OUT. w and x 16-byte aligned, Kd a multiple of 8.
 *  ws       fp32 split-K scratch of at least *ws_floats elements (may be NULL
 *           when *ws_floats is 0), tickets int32 [*n_tickets] that must be
 *           zero before the first call; the kernel leaves them zero again.
 * pe_linear_scratch reports the sizes for a shape on the current device. */
int pe_linear_scratch(int32_t dtype, int32_t M, int32_t N, int32_t Kd, int64_t* ws_floats, int32_t* n_tickets);
int pe_linear(int32_t dtype, int32_t M, int32_t N, int32_t Kd, const void* w, const void* x, float* y,
              float* ws, int32_t* tickets, void* stream);
/* The FP8-weight GEMM engine on its own: y[n, m] = scale[m] * sum_k q[m, k] * x[n, k]
 *  w  [M, Kd] E4M3 codes (uint8), w_scale [M] fp32, x [N, Kd] bf16, y [N, M]
 *  fp32 OUT; Kd a multiple of 16, w and x 16-byte aligned. ws / tickets as
 *  for pe_linear, sized by pe_linear_scratch(PE_DTYPE_FP8W, ...). */
int pe_linear_fp8(int32_t M, int32_t N, int32_t Kd, const void* w, const float* w_scale, const void* x, float* y,
                  float* ws, int32_t* tickets, void* stream);

/* pe_linear for callers that cannot allocate device memory (this entry point
 * has no counterpart in the method's description). Some callers may not call cudaMalloc
 * where they run a GEMM: code running while another thread captures a CUDA
 * graph in global capture mode, where cudaMalloc is prohibited, or runtimes
 * whose device memory is fully reserved by their own allocator. This variant
 * computes the same y[n, m] = sum_k w[m, k] * x[n, k] as pe_linear (same
 * arguments minus ws / tickets) but keeps its split-K scratch in fixed arrays
 * inside the library: 8 MiB of partials and 4096 tickets per device, held
 * until the process exits. It allocates nothing.
 *  - Shapes whose plan needs more scratch than that (pe_linear_scratch
 *    reports the need: more than 2 Mi floats, or more than 4096 tickets
 *    when it needs tickets at all) return PE_ERR_ARG with a message giving
 *    the need and the maximum, before any launch (pe_linear has no limit).
 *  - The first call on each device looks up the arrays' device addresses
 *    (cudaGetSymbolAddress) with that device current and loads the kernel
 *    of both dtypes; make that first call (in either dtype) before any
 *    stream capture that should contain later calls, or that runs while
 *    later calls are made. After cudaDeviceReset the cached addresses are
 *    stale: do not call it on that device again in the same process.
 *  - Every call on a device shares the same arrays: calls that can overlap
 *    on the GPU (several streams or host threads) race and must be serialised
 *    by the caller. Each call clears the tickets it uses on its stream. */
int pe_linear_noalloc(int32_t dtype, int32_t M, int32_t N, int32_t Kd, const void* w, const void* x, float* y,
                      void* stream);

/* Linear layer with 4-bit weights and group scales, for the few token rows of
 * a draft pass (beside pe_linear_fp8):
 *   y[n, m] = sum_k (c[m, k] - z[m, k / group]) * s[m, k / group] * x[n, k]
 *  w       [M, Kd/2] uint8: code c (0..15) of column 2i in the low half of byte i, of 2i+1 in the high half
 *  w_scale [M, ceil(Kd/group)] of scale_dtype (PE_DTYPE_BF16 or PE_DTYPE_FP32); w_zero the same shape, uint8
 *          (0..255), or NULL: every zero point is 8
 *  x       [N, Kd] bf16, rows ld_x elements apart; y [N, M] fp32 OUT, rows ld_y apart
 * group is 32, 64 or 128 (the last group of a row may be short); Kd a
 * multiple of 32; w and x 16-byte aligned, w_scale and y to their elements,
 * ld_x a multiple of 8. Products and sums in fp32; the weights are not rounded,
 * x only where it is below 2^-28 of the largest value of its 256 columns. Scales
 * of magnitudes up to 2^96: x is shifted by powers of two so that a group's sum
 * can stand at 2^31, and its product with the scale has to be finite. A row of
 * x that holds an infinity or NaN gives infinities or NaN in its row of y, and
 * in no other. No scratch; the device that holds the tensors must be current.
 * Rows of x go 8 or 16 at a time, and each of these reads and decodes the
 * weights again: from some 32 rows on pe_linear_fp8 is quicker. N <= 524280. */
int pe_linear_w4(int32_t M, int32_t N, int32_t Kd, int32_t group, const uint8_t* w, int32_t scale_dtype,
                 const void* w_scale, const uint8_t* w_zero, const void* x, int64_t ld_x, float* y, int64_t ld_y,
                 void* stream);

/* Pages for a growing batch, on the device (no host round trip between a
 * verify and the next pass): request b holds page_counts[b] pages, the first
 * entries of its page_table row, and seq_lens[b] committed entries, and is to
 * take new_lens[b] more. What is missing comes from the top of a stack of free
 * pages (free_pages[0 .. free_count)), in request order.
 *  seq_lens, new_lens, page_counts [B] int32; new_lens in 0..n_max
 *  page_table   [B, max_pages] int32 in/out: entries page_counts[b] .. are written
 *  free_pages   [free_cap] int32, free_count [1] int32
 *  page_counts_out [B], free_count_out [1] OUT; must not alias their inputs
 *  slot_mapping [B, n_max] int32 OUT: slot (page*16 + offset) of entries
 *               S_b .. S_b+n_b-1, then -1
 *  status       [B] OUT: PE_REQ_BAD_INPUT (a length out of range, or fewer
 *               pages than seq_lens needs), PE_REQ_CAPACITY (max_pages, or the
 *               stack runs out: this request and every later one that needs
 *               pages get none), PE_REQ_BAD_PAGE (a page of the new entries is
 *               outside [0, num_pages); the pages it took stay with it). The
 *               slots of a request that is not OK are -1. */
int pe_assign_pages(int32_t B, const int32_t* seq_lens, const int32_t* new_lens, const int32_t* page_counts,
                    int32_t* page_counts_out, int32_t* page_table, int32_t max_pages, int32_t num_pages,
                    const int32_t* free_pages, int32_t free_cap, const int32_t* free_count, int32_t* free_count_out,
                    int32_t n_max, int32_t* slot_mapping, int32_t* status, void* stream);

/* The way back: request b keeps the pages of its first keep_lens[b] entries
 * (0: it is finished) and pushes the others, in request and page order, onto
 * the stack; their page_table entries become -1. page_counts_out and
 * free_count_out may alias their inputs. status: PE_REQ_BAD_INPUT (keep_lens
 * beyond the request's pages), PE_REQ_BAD_PAGE (one of the pages is outside
 * [0, num_pages)), PE_REQ_CAPACITY (the stack is full: this request and every
 * later one keep theirs); a request that is not OK keeps everything. */
int pe_release_pages(int32_t B, const int32_t* keep_lens, const int32_t* page_counts, int32_t* page_counts_out,
                     int32_t* page_table, int32_t max_pages, int32_t num_pages, int32_t* free_pages, int32_t free_cap,
                     const int32_t* free_count, int32_t* free_count_out, int32_t* status, void* stream);

/* A paged KV cache in 8 bits, half the bytes of the bf16 one:
 *  k_codes, v_codes [num_pages][nkv][16][hd] uint8: E4M3 codes
 *  k_scale, v_scale [num_pages][nkv] fp32: entry = code * scale of its page and head
 * One layer's cache; the layers of a model are as many of them.
 *
 * pe_kv8_append stores rows[b] (NULL: n_max) new rows of request b at its
 * entries S_b, S_b+1, ...:
 *  k, v  [B, n_max, nkv, hd] bf16, rows ld_k / ld_v elements apart (columns of
 *        a fused projection's output will do); rows past rows[b] are not read
 *  status [B] OUT; a request that is not OK writes nothing.
 * The scale of a page and head is the smallest power of two (2^-126 at least)
 * under which the new rows' largest finite magnitude is at most 448; codes are
 * the nearest (ties to even). A page with committed entries keeps its scale if
 * that is larger; if not, their codes are moved to the new one. Infinities
 * become +-448, a NaN the NaN code. Nothing else of the cache is touched;
 * codes behind the last new row keep their bytes. A page never returns to a
 * smaller scale while it has committed entries, also where the larger one came
 * from rows that were rejected since. Pages that two requests share, or that
 * stand in a row of the table twice, must be full: two appends to one page race.
 * k, v 8-byte aligned, ld_k and ld_v multiples of 4, codes 16-byte aligned. */
int pe_kv8_append(int32_t B, int32_t n_max, int32_t nkv, int32_t hd, const void* k, int64_t ld_k, const void* v,
                  int64_t ld_v, const int32_t* seq_lens, const int32_t* rows, const int32_t* page_table,
                  int32_t max_pages, int32_t num_pages, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
                  float* v_scale, int32_t* status, void* stream);

/* Attention of the K rows of each request over that cache: row j < rows[b]
 * (NULL: K) of request b attends to entries 0 .. S_b + j (its own row is
 * appended before), query head h over kv head h / (nq/nkv), softmax of
 * scale * q.k in fp32.
 *  q      [B, K, nq, hd] bf16, rows ld_q elements apart
 *  out    [B, K, nq, hd] bf16 OUT, rows ld_out apart; rows past rows[b], and
 *         all rows of a request that is not OK, are zero
 *  ws     scratch of pe_attention_kv8_scratch floats (two partial results of
 *         up to 128 rows for each multiprocessor, 20 MB at most, whatever
 *         max_pages is), 16-byte aligned; needs no initial value, and calls
 *         that can overlap need one each
 *  status [B] OUT; a page-table entry of a needed page that is outside
 *         [0, num_pages) is PE_REQ_BAD_PAGE
 * K * (nq/nkv) <= 128, hd 64 or 128; q, out and codes 16-byte aligned, ld_q and
 * ld_out multiples of 8; B * nkv * (max_pages + 32) < 2^30.
 * Entries that no row sees may hold anything. A NaN code of K makes the rows
 * that see its entry NaN, one of V that dimension of them (all of them where
 * the entry stands in a page that some row does not see whole, or within three
 * pages of one), and neither any other row. A row of q that holds an infinity
 * or a NaN is NaN.
 * Rounded to fewer than 32 bits, besides the output: the weights times their
 * page's V scale, to fp16 relative to the row's largest such product (2^-11 of
 * each; products below 2^-19 of the largest: 2^-30 of it), and the queries.
 * Up to 8 rows for a kv head, K * (nq/nkv) (64-wide heads: 16), a value of q is
 * off by 2^-25 of its row's largest at most and exact from 2^-17 of that on;
 * with more rows by 2^-17 of the largest, and exact from 2^-9 of it on. */
int pe_attention_kv8_scratch(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int32_t max_pages, int64_t* ws_floats);
int pe_attention_kv8(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const void* q,
                     int64_t ld_q, const int32_t* seq_lens, const int32_t* rows, const int32_t* page_table,
                     int32_t max_pages, int32_t num_pages, const uint8_t* k_codes, const uint8_t* v_codes,
                     const float* k_scale, const float* v_scale, float scale, void* out, int64_t ld_out, float* ws,
                     int64_t ws_floats, int32_t* status, void* stream);

/* A paged KV cache in 4 bits, about half the bytes of the 8-bit one:
 *  k_codes, v_codes   [num_pages][nkv][16][hd/2] uint8: code n (0..15) of dimension 2i in the low half of byte i, of
 *                     2i+1 in the high half
 *  k_params, v_params [num_pages][nkv][16][2] bf16: scale and base of an entry; value = base + scale * n
 * One layer's cache; the layers of a model are as many of them.
 *
 * pe_kv4_append turns new query and key rows to their positions and stores
 * keys and values: rows[b] (NULL: n_max) new rows of request b at its entries
 * S_b, S_b+1, ...
 *  q, k, v [B, n_max, heads, hd] bf16, rows ld_* elements apart (columns of a
 *          fused projection's output will do); rows past rows[b] are not read.
 *          n_q_heads may be 0 (q and q_out are then not read)
 *  rope_theta: row j of request b has position p = positions[b] + j (positions
 *          NULL: S_b + j), and dimensions i and i + hd/2 of a head of q or k turn
 *          by p * rope_theta^(-2i/hd); 0: nothing is turned. Otherwise at least 1
 *  q_out   [B, n_max, nq, hd] bf16 OUT, rows ld_q_out apart (may be q itself):
 *          the turned queries; zero past rows[b] and in requests that are not OK
 *  status  [B] OUT; a request that is not OK writes nothing else.
 *          PE_REQ_BAD_INPUT: a length or position below 0 or rows[b] above n_max
 * Of the values x of a head of a row: base = bf16(min x), scale = bf16(max(max x -
 * base, 0) / 15), n the nearest (ties to even) to (x - base) / scale in 0..15, 0
 * where scale is 0. A turned key is not rounded before. Angles are off by 2^-33
 * of a turn at most at every position, sines and cosines are fp32. A head of a
 * row that holds an infinity or NaN, or whose largest value and base lie 2^128 or
 * more apart, stands as NaN (scale and base). An entry depends on its row alone;
 * nothing else of the cache is touched. Requests whose new entries are the same
 * places of the cache race. q_out over q has q's row stride; otherwise no output
 * shares memory with an input.
 * q, k, v and q_out 8-byte aligned, their strides multiples of 4, the cache's
 * arrays 16-byte aligned. */
int pe_kv4_append(int32_t B, int32_t n_max, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const void* q,
                  int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, float rope_theta,
                  const int32_t* positions, const int32_t* seq_lens, const int32_t* rows, const int32_t* page_table,
                  int32_t max_pages, int32_t num_pages, uint8_t* k_codes, uint8_t* v_codes, void* k_params,
                  void* v_params, void* q_out, int64_t ld_q_out, int32_t* status, void* stream);

/* Attention of the K rows of each request over that cache, with the arguments
 * of pe_attention_kv8 (k_params and v_params in the place of the scales, the
 * cache's arrays 16-byte aligned) and its rules for rows, masks, scratch (of
 * pe_attention_kv4_scratch floats), pages and status. out shares no memory with q.
 * Entries that no row sees may hold anything. An entry whose parameters are not
 * finite makes the rows that see it NaN, and no other row; one that a row does
 * not see does not move it, whatever its size. A row of q that holds an infinity
 * or a NaN is NaN. Scales are not negative, and values of V times the entries that
 * a row sees stay below 2^119: sums are of weights up to 2^8. Scores may be of any
 * size that fp32 holds. Below 2^-104 scales of V have fewer bits in the products.
 * Rounded to fewer than 32 bits, besides the output: the queries, to fp16 under a
 * power of two of their row (a value is off by 2^-25 of its row's largest at
 * most), and the weights times V's scale, to fp16 relative to the row's largest
 * such product (2^-11 of each; small ones by 2^-26 of the largest). With more than
 * 16 rows for a kv head, K * (nq/nkv), also K and V, to fp16 under a power of two
 * of their page where every row sees the unit of 64 entries that it stands in:
 * 2^-11 of a value of K, 2^-10 of scale |n - 8| + |base + 8 scale| for V, and
 * 2^-18 of the page's largest K, 2^-36 of its largest V. */
int pe_attention_kv4_scratch(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int32_t max_pages, int64_t* ws_floats);
int pe_attention_kv4(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const void* q,
                     int64_t ld_q, const int32_t* seq_lens, const int32_t* rows, const int32_t* page_table,
                     int32_t max_pages, int32_t num_pages, const uint8_t* k_codes, const uint8_t* v_codes,
                     const void* k_params, const void* v_params, float scale, void* out, int64_t ld_out, float* ws,
                     int64_t ws_floats, int32_t* status, void* stream);

/* What rows of logits say of given tokens (beside pe_sample_drafts and
 * pe_verify_stochastic): with p = softmax(logits / temperature) of a row,
 *  logits       [R, V] bf16 or fp32 (dtype: PE_DTYPE_BF16 or PE_DTYPE_FP32), rows ld elements apart
 *               (0: one row, of which several tokens are asked)
 *  tokens       [R] int32
 *  logprobs     [R] fp32 OUT: ln p[tokens[r]] (NaN for a token outside [0, V))
 *  entropy      [R] fp32 OUT or NULL: -sum p ln p
 *  top_tokens   [R, top] int32 OUT, top_logprobs [R, top] fp32 OUT: the top
 *               likeliest tokens in order, of equal ones the lower index first
 *               (top 0..32, at most V; NULL where it is 0), and ln p of each
 * A logit of -inf is a token that cannot be (ln p = -inf, and it adds nothing to
 * the entropy); -FLT_MAX is one like any other (ln p below fp32's range is -inf). A row that holds a NaN or +inf,
 * or only -inf, has no probabilities: NaN in the place of each, NaN logits
 * ordered behind all others. The temperature lies in 2^-63 .. 2^64, R and V are 2^30 at most; a finite
 * logit over it has a magnitude up to 2^120, or the logit is -FLT_MAX. Sums in
 * fp32, each weight off by about 2^-21 of itself. No output shares memory with an
 * input. */
int pe_token_logprobs(int32_t R, int32_t V, int32_t dtype, const void* logits, int64_t ld, const int32_t* tokens,
                      float temperature, float* logprobs, float* entropy, int32_t top, int32_t* top_tokens,
                      float* top_logprobs, void* stream);

/* One whole step (pe_draft, then pe_verify_rebuild on its drafts) captured
 * once into a CUDA graph and replayed with a single launch. The arguments are
 * those of pe_draft and pe_verify_rebuild (drafts are shared; draft_status and
 * verify_status are the two status arrays); every pointer is baked into the
 * graph, so callers update buffer CONTENTS between launches, not addresses.
 * When positions_out/seq_lens_out alias positions/seq_lens, each replay
 * advances the batch metadata in place. Creation synchronises nothing and
 * enqueues nothing; launches are asynchronous on `stream`. */
typedef struct pe_step_graph pe_step_graph;
int pe_step_graph_create(pe_handle* h, int32_t B, int32_t K, const int32_t* last_token, const void* target_hidden,
                         const int32_t* positions, const int32_t* seq_lens, const int32_t* page_table,
                         int32_t max_pages, int32_t num_pages, void* k_cache, void* v_cache, int32_t* drafts,
                         int32_t* draft_status, const int32_t* target_tokens, int32_t* positions_out,
                         int32_t* seq_lens_out, int32_t* accepted, int32_t* bonus, int32_t* emitted,
                         int32_t* slot_mapping, int32_t* rollback_slots, int32_t* verify_status,
                         pe_step_graph** out);
/* The same with the draft half chosen by draft_mode: PE_DRAFT_PARALLEL
 * (pe_draft, what pe_step_graph_create captures) or PE_DRAFT_SEQUENTIAL
 * (pe_draft_sequential). */
#define PE_DRAFT_PARALLEL   0
#define PE_DRAFT_SEQUENTIAL 1
int pe_step_graph_create_ex(pe_handle* h, int32_t draft_mode, int32_t B, int32_t K, const int32_t* last_token,
                            const void* target_hidden, const int32_t* positions, const int32_t* seq_lens,
                            const int32_t* page_table, int32_t max_pages, int32_t num_pages, void* k_cache,
                            void* v_cache, int32_t* drafts, int32_t* draft_status, const int32_t* target_tokens,
                            int32_t* positions_out, int32_t* seq_lens_out, int32_t* accepted, int32_t* bonus,
                            int32_t* emitted, int32_t* slot_mapping, int32_t* rollback_slots,
                            int32_t* verify_status, pe_step_graph** out);
int pe_step_graph_launch(pe_step_graph* g, void* stream);
/* kernels one replay launches */
int pe_step_graph_launch_count(const pe_step_graph* g);
void pe_step_graph_destroy(pe_step_graph* g);

/* Synchronise `stream` and return (then clear) the device error word of h
 * (PE_DEVERR_* bits; 0 = no device-side wait gave up). */
int pe_device_errors(pe_handle* h, void* stream, uint32_t* out_bits);

/* Test support for the bounded-wait give-up path (no counterpart in the
 * method's description; host-side fault injection, nothing on the device is made to fault).
 * Enqueues on `stream` a write that primes the arrival tickets of the first
 * phase of the handle's persistent layer chain so that its shared tiles never
 * complete. The next pe_draft's chain launches then wait for a phase that
 * never finishes: each such wait gives up after its time limit (1 s), sets
 * PE_DEVERR_CHAIN_TIMEOUT, and the kernel returns; its outputs for that call
 * are meaningless. The chain resets its tickets and counters on the way out,
 * so the handle is usable again once pe_device_errors has read and cleared
 * the error word. Returns PE_ERR_UNSUPPORTED when the handle runs no chain
 * (it runs one when created with PE_LAYER_CHAIN=1 in the environment, bf16,
 * for draft passes of at most 64 rows). */
int pe_test_stall_chain(pe_handle* h, void* stream);

/* The same for pe_attention_kv8: the next call in this process that goes by its
 * tensor-memory kernel (more than 8 query rows of a kv head, 64-wide heads more
 * than 16) has every barrier of one kind (1: K codes, 2: V tiles, 3: weights)
 * wait for one arrival more than there are, so its waits give up after their
 * limit (1 s) and the call reports PE_REQ_TIMEOUT. Later calls are not touched. */
int pe_test_stall_attention_kv8(int32_t barrier);
/* And for pe_attention_kv4 (its tensor-memory kernel: more than 16 query rows of a kv head). */
int pe_test_stall_attention_kv4(int32_t barrier);

/* Kernel kinds of the draft pass, for launch accounting and profiling. */
#define PE_KERNEL_FC         0
#define PE_KERNEL_ROW_BUILD  1
#define PE_KERNEL_RMSNORM    2   /* reserved: RMSNorm is folded into the GEMM epilogues and never launched */
#define PE_KERNEL_QKV        3
#define PE_KERNEL_ATTENTION  4   /* with length-aware pieces also the merge kernel that follows it */
#define PE_KERNEL_O_PROJ     5
#define PE_KERNEL_GATE_UP    6
#define PE_KERNEL_DOWN       7
#define PE_KERNEL_LM_HEAD    8
#define PE_KERNEL_ARGMAX     9
#define PE_KERNEL_LAYER_CHAIN 10  /* O, gate/up, down and the next QKV (or the LM head) in one persistent launch */
#define PE_KERNEL_COUNT      11

/* Measurement hook: after pe_profile_start, every launch of `kernel_kind`
 * made by pe_draft (up to max_launches of them) is bracketed by CUDA events
 * recorded on the launch stream; an attention that runs as length-aware
 * pieces is bracketed together with its merge kernel (one interval per
 * layer). pe_profile_stop waits for those events and returns the summed
 * device time (ms) and the number of intervals timed. */
int pe_profile_start(pe_handle* h, int32_t kernel_kind, int32_t max_launches);
int pe_profile_stop(pe_handle* h, float* total_ms, int32_t* launches);
const char* pe_kernel_name(int32_t kind);

/* Number of kernels the last pe_draft call enqueued (for launch accounting;
 * merge kernels included). */
int pe_last_launch_count(const pe_handle* h);

void pe_destroy(pe_handle* h);

/* Thread-local description of the last error (never NULL). */
const char* pe_last_error(void);

int pe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* PE_H */
