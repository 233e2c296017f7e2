/*
 * qmoe.h -- C ABI of the GB300 (sm_103a) qwen3moe Mixture-of-Experts FFN over
 * GGUF k-quant expert weights.
 *
 * The operation (aprender issue "qwen3moe (Qwen3-30B-A3B, Qwen3-Coder-30B-A3B,
 * Q4_K_M) has NO working CUDA path", sections "File facts" and "Gaps ... G3"):
 *
 *   logits = Wr x (+ bias)                        F32 router GEMV [E x H]
 *   S, w   = top-k(softmax(logits)), renormalised  ("softmax, top-8, renorm")
 *   for each selected expert e (addressed in place as base + e * stride):
 *     g = Wg_e x, u = Wu_e x                      Q4_K gate / up dequant-GEMV
 *     a = silu(g) * u                             fused SwiGLU
 *     y_e = Wd_e a                                Q6_K or Q4_K down dequant-GEMV
 *   out = residual + sum_j w_j y_{S_j}            weighted sum into the residual
 *
 * qmoe_forward_q8k runs the same layer with x and a quantised to 8-bit (Q8_K)
 * activations before every expert GEMV (the int8 variant of "Gaps ... G8").
 * qmoe_forward_fp8 and qmoe_forward_nvfp4 run it over FP8 block-scaled and
 * NVFP4 experts instead of k-quants (qmoe_nvfp4_quantize makes NVFP4 weights
 * from BF16 ones).
 * qmoe_rmsnorm, qmoe_fp8_quantize, qmoe_linear_fp8, qmoe_rope and
 * qmoe_kv4_append_rope are what a decoder layer over FP8 weights needs around
 * qmoe_forward_fp8 and the paged cache (qmoe_kv4_*).
 *
 * Conventions shared by every entry point:
 *  - Every tensor pointer is a DEVICE pointer that the caller allocated and owns
 *    (except qmoe_forward_host, whose activations are host pointers).  The
 *    library never copies, repacks or frees caller memory.
 *  - Quantised tensors are raw GGUF superblocks: Q4_K = 144 B per 256 weights
 *    (fp16 d, fp16 dmin, 12 B packed 6-bit scales/mins, 128 B nibbles); Q6_K =
 *    210 B per 256 weights (128 B ql, 64 B qh, 16 int8 scales, fp16 d).  A
 *    matrix with R outputs and C inputs is R rows of C/256 consecutive
 *    superblocks; expert e of a 3-D expert tensor starts at
 *    base + e * R * (C/256) * block_bytes.
 *  - F32 activations are row-major [n_tokens][hidden].
 *  - Work is enqueued asynchronously on the context's stream; no call below
 *    synchronises the host, allocates memory or copies weights, except
 *    qmoe_create / qmoe_destroy (allocate / free the workspace),
 *    qmoe_forward_host (copies activations and synchronises) and
 *    qmoe_get_status (synchronises).
 *  - Errors are returned as qmoe_status; no exception crosses the ABI.
 *    Argument errors are detected on the host before anything is enqueued.
 *    qmoe_last_error() gives a one-line description of the last failure.
 *  - A context is not thread-safe: one host thread at a time, and calls that
 *    share a context must be ordered on its stream (they share the workspace).
 */
#ifndef QMOE_H
#define QMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QMOE_OK = 0,
    QMOE_ERR_INVALID_ARG = 1,       /* null pointer, bad size or count */
    QMOE_ERR_MISALIGNED = 2,        /* a base pointer is not 16-byte aligned */
    QMOE_ERR_UNSUPPORTED_QTYPE = 3, /* qtype not allowed for that tensor */
    QMOE_ERR_SHAPE = 4,             /* hidden/ffn not a multiple of 256, n_tokens > max */
    QMOE_ERR_NO_MEMORY = 5,         /* workspace does not fit; message names the bytes */
    QMOE_ERR_CUDA = 6,              /* a CUDA runtime call failed; message names it */
    QMOE_ERR_TIMEOUT = 7,           /* a bounded device-side wait gave up */
    QMOE_ERR_DEVICE_CHECK = 8       /* a device-side index check failed */
} qmoe_status;

typedef enum { QMOE_Q4_K = 1, QMOE_Q6_K = 2 } qmoe_qtype;

typedef struct qmoe_ctx qmoe_ctx;

/* Geometry fixed at create time.  The MoE part (hidden, n_experts, top_k, ffn)
 * is required; the attention part is needed only by qmoe_decode_step and may
 * be all zero otherwise (Qwen3-30B-A3B: 32 q heads, 4 kv heads, head_dim 128,
 * rope base 1e7, RMSNorm eps 1e-6; head_dim is NOT hidden / n_heads -- aprender
 * issue "Qwen3 GPU inference produces garbage output", "Fix Applied"). */
typedef struct {
    int hidden;          /* H, multiple of 256 */
    int n_experts;       /* E, 1..1024 */
    int top_k;           /* k, 1..min(E, 16) */
    int ffn;             /* F, expert FFN width, multiple of 256 */
    int norm_topk_prob;  /* 1: renormalise the k selected probabilities (qwen3moe) */
    int max_tokens;      /* largest n_tokens any call will pass (workspace size) */
    int n_heads;         /* attention q heads (decode step only, else 0) */
    int n_kv_heads;      /* attention kv heads, divides n_heads */
    int head_dim;        /* 128 for qwen3moe (a multiple of 64, <= 256) */
    int max_ctx;         /* KV-cache positions per layer, 1..262144 */
    float rope_base;     /* NEOX RoPE base */
    float rms_eps;       /* RMSNorm epsilon (all four norms) */
    void* stream;        /* cudaStream_t the work is enqueued on (NULL = legacy default) */
} qmoe_config;

/* Create a context on the current CUDA device and allocate its workspace
 * (router logits, expert ids / weights, per-expert pair lists, intermediate
 * activations, all sized by max_tokens).  Returns QMOE_ERR_NO_MEMORY with a
 * message giving the bytes needed and free, instead of failing later.
 * On success *out owns the workspace until qmoe_destroy. */
qmoe_status qmoe_create(const qmoe_config* cfg, qmoe_ctx** out);

/* Free the workspace (synchronises the context's stream first).  NULL is a no-op. */
void qmoe_destroy(qmoe_ctx* ctx);

/* Change the stream later calls enqueue on. */
qmoe_status qmoe_set_stream(qmoe_ctx* ctx, void* stream);

/* hidden_out = hidden_in + MoE(hidden_in) for n_tokens tokens.
 *  hidden_in, hidden_out : F32 [n_tokens][H] (device).  They may alias only
 *                          when n_tokens <= 8 (decode); otherwise -> INVALID_ARG.
 *  router_w              : F32 [E][H] (device), the ffn_gate_inp tensor.
 *  gate_exps, up_exps    : [E][F rows][H/256 superblocks], Q4_K (or Q6_K).
 *  down_exps             : [E][H rows][F/256 superblocks], Q6_K or Q4_K.
 *  All base pointers 16-byte aligned.  n_tokens in 1..max_tokens.
 * Expert ids are selected on the F32 logits, ties to the lower index. */
qmoe_status qmoe_forward(qmoe_ctx* ctx, const float* hidden_in, const float* router_w,
                         const void* gate_exps, const void* up_exps, const void* down_exps,
                         qmoe_qtype gate_t, qmoe_qtype up_t, qmoe_qtype down_t,
                         int n_tokens, float* hidden_out);

/* General form:  out = residual + MoE(ffn_in), router logits += router_bias.
 *  residual     : F32 [n_tokens][H] or NULL (then residual = ffn_in).
 *  router_bias  : F32 [E] or NULL.
 *  ids_out      : int32 [n_tokens][k] or NULL -- selected experts, ordered by
 *                 descending logit (ties: lower index first).
 *  weights_out  : F32 [n_tokens][k] or NULL -- their routing weights.
 * out may alias residual (not ffn_in) when n_tokens <= 8. */
qmoe_status qmoe_forward_ex(qmoe_ctx* ctx, const float* ffn_in, const float* residual,
                            const float* router_bias, const float* router_w,
                            const void* gate_exps, const void* up_exps, const void* down_exps,
                            qmoe_qtype gate_t, qmoe_qtype up_t, qmoe_qtype down_t,
                            int n_tokens, float* out, int32_t* ids_out, float* weights_out);

/* The same layer with 8-bit activations in every expert GEMV: the int8 (DP4A)
 * variant of the aprender issue "qwen3moe (Qwen3-30B-A3B, ...) has NO working
 * CUDA path" ("Gaps ... G8"; its R1 receipt measures it against FP32
 * activations).  hidden_out = hidden_in + MoE(hidden_in) where x (per token)
 * and the SwiGLU output (per selected expert) are first quantised to Q8_K
 * blocks of 256 values: fp32 scale d, int8 codes, the block's largest-magnitude
 * value (first on a tie) on code -128 (s = -128/v, q = min(127, rint(s*x)),
 * d = 1/s, fp32), and each weight row is dotted with the codes in integer form.
 * The router stays F32.  Arguments as qmoe_forward; ids_out / weights_out as
 * qmoe_forward_ex (nullable).  hidden_out may alias hidden_in.  Any n_tokens in
 * 1..max_tokens; hidden and ffn multiples of 256 (as for every entry point).
 * Argument errors are returned before any launch, as for qmoe_forward. */
qmoe_status qmoe_forward_q8k(qmoe_ctx* ctx, const float* hidden_in, const float* router_w,
                             const void* gate_exps, const void* up_exps, const void* down_exps,
                             qmoe_qtype gate_t, qmoe_qtype up_t, qmoe_qtype down_t,
                             int n_tokens, float* hidden_out, int32_t* ids_out, float* weights_out);

/* The MoE layer over FP8 block-scaled experts with the F32 router (atlasinference
 * source page "spark_model/weight_loader/qwen3.rs", load_layers: experts kept as
 * FP8 with one scale per 128 x 128 block, FP8 weights against wider
 * activations, and the option of a full-precision router so that expert
 * selection is not decided by quantised logits).
 *   gate_exps / up_exps: E4M3 ("e4m3fn") codes [E][ffn][hidden], one byte each;
 *   down_exps: codes [E][hidden][ffn];
 *   gate_scale / up_scale: fp32 [E][ffn/128][hidden/128];
 *   down_scale: fp32 [E][hidden/128][ffn/128];
 *   weight (r, c) of expert e = e4m3(code) * scale[e][r/128][c/128].
 * Codes 0x7F / 0xFF (NaN) are not valid weights.  Up to 32 tokens the expert
 * GEMVs run on the CUDA cores with x, the SwiGLU output and every sum in fp32;
 * more tokens run as grouped GEMMs on the tensor cores (weights widened to fp16
 * as e4m3 * scale rounded once, x and the SwiGLU output rounded to fp16, fp32
 * accumulation), like the k-quant path of qmoe_forward.  hidden_out = hidden_in + MoE(hidden_in); it may alias
 * hidden_in for any n_tokens.  ids_out / weights_out as qmoe_forward_ex
 * (nullable).  Serves hidden/256 in {2, 4, 8, 16} and ffn/256 in 1..6
 * (QMOE_ERR_SHAPE otherwise).  Code and activation pointers 16-byte aligned,
 * scale pointers 4-byte aligned (QMOE_ERR_MISALIGNED).  Argument errors are
 * returned before any launch. */
qmoe_status qmoe_forward_fp8(qmoe_ctx* ctx, const float* hidden_in, const float* router_w,
                             const void* gate_exps, const float* gate_scale,
                             const void* up_exps, const float* up_scale,
                             const void* down_exps, const float* down_scale,
                             int n_tokens, float* hidden_out, int32_t* ids_out,
                             float* weights_out);

/* The MoE layer over NVFP4 experts with the F32 router (atlasinference source
 * page "spark_model/weight_loader/qwen3.rs", load_layers: weights quantised
 * from BF16 to NVFP4 at load).  NVFP4 (the public format): FP4 E2M1 elements,
 * two per byte with the even element in the low nibble, one E4M3 scale per 16
 * consecutive elements of a row, one fp32 scale per matrix:
 *   weight (r, c) of expert e = e2m1(code) * e4m3(bscale[e][r][c/16]) * global[e].
 *   gate_exps / up_exps: codes [E][ffn][hidden/2]; *_bscale [E][ffn][hidden/16];
 *   down_exps: codes [E][hidden][ffn/2]; down_bscale [E][hidden][ffn/16];
 *   *_global: fp32 [E].
 * Up to 32 tokens (and whenever a block-scale pointer is not 16-byte aligned)
 * the expert GEMVs run on the CUDA cores with x, the SwiGLU output and every
 * sum in fp32; more tokens run as grouped GEMMs on the tensor cores (weights
 * widened to fp16 as e2m1 * e4m3 * global rounded once, x and the SwiGLU
 * output rounded to fp16, fp32 accumulation).  hidden_out = hidden_in + MoE(hidden_in) and may alias
 * hidden_in.  ids_out / weights_out as qmoe_forward_ex (nullable).  Serves
 * hidden/512 in {1, 2, 4, 8} and ffn/256 in 1..6 (QMOE_ERR_SHAPE otherwise).
 * Code and activation pointers 16-byte aligned, block scales 2-byte, globals
 * 4-byte (QMOE_ERR_MISALIGNED).  Argument errors are returned before any launch. */
qmoe_status qmoe_forward_nvfp4(qmoe_ctx* ctx, const float* hidden_in, const float* router_w,
                               const void* gate_exps, const void* gate_bscale,
                               const float* gate_global, const void* up_exps,
                               const void* up_bscale, const float* up_global,
                               const void* down_exps, const void* down_bscale,
                               const float* down_global, int n_tokens, float* hidden_out,
                               int32_t* ids_out, float* weights_out);

/* Runtime quantisation of n_mats consecutive BF16 matrices [rows][cols] (device
 * memory, bit patterns) to NVFP4 (same page: a global-absmax pass, then the
 * per-block quantisation).  Per matrix, every decision in fp32:
 *   amax = max |x|; global = amax / 2688 (448 * 6);
 *   per 16 elements: s = E4M3 nearest to bmax / (6 * global) (ties to even,
 *   saturating at 448); d = e4m3(s) * global; code = E2M1 nearest to x / d
 *   (ties to even, saturating at 6; 0 where d = 0).
 * Outputs (device, caller-owned): codes [n_mats][rows][cols/2] (8-byte
 * aligned), bscale [n_mats][rows][cols/16], global [n_mats] (4-byte aligned).
 * x 16-byte aligned; cols a positive multiple of 16; n_mats in 1..1024.
 * Enqueued on the context's stream; uses a few bytes of its workspace, so it is
 * ordered with the context's other calls. */
qmoe_status qmoe_nvfp4_quantize(qmoe_ctx* ctx, const void* x_bf16, int n_mats, int rows, int cols,
                                void* codes, void* bscale, float* global);

/* Same as qmoe_forward, but hidden_in / hidden_out are HOST pointers (pinned
 * memory gives asynchronous copies).  Copies the activations to the device
 * workspace, runs the layer, copies the result back and synchronises the
 * stream before returning.  Weights stay device pointers. */
qmoe_status qmoe_forward_host(qmoe_ctx* ctx, const float* hidden_in_host, const float* router_w,
                              const void* gate_exps, const void* up_exps, const void* down_exps,
                              qmoe_qtype gate_t, qmoe_qtype up_t, qmoe_qtype down_t,
                              int n_tokens, float* hidden_out_host);

/* Weights of one qwen3moe decoder layer (all device pointers). */
typedef struct {
    const float* attn_norm;  /* [H] input RMSNorm weight */
    const void* wq;          /* [n_heads*head_dim rows][H], Q4_K */
    const void* wk;          /* [n_kv*head_dim rows][H], Q4_K */
    const void* wv;          /* [n_kv*head_dim rows][H], Q4_K */
    const void* wo;          /* [H rows][n_heads*head_dim], Q4_K */
    const float* q_norm;     /* [head_dim] per-head Q RMSNorm weight */
    const float* k_norm;     /* [head_dim] per-head K RMSNorm weight */
    const float* ffn_norm;   /* [H] post-attention RMSNorm weight */
    const float* router_w;   /* [E][H] F32 */
    const void* gate_exps;   /* MoE experts as in qmoe_forward */
    const void* up_exps;
    const void* down_exps;
    qmoe_qtype down_t;       /* Q6_K or Q4_K (per layer) */
    void* k_cache;           /* fp16 [n_kv][max_ctx][head_dim]; slot pos is written */
    void* v_cache;           /* fp16 [n_kv][max_ctx][head_dim]; slot pos is written */
} qmoe_layer_weights;

/* One batch-1 decode step through n_layers qwen3moe decoder layers, in place on
 * hidden (F32 [H], device).  Per layer: x = RMSNorm(h)*attn_norm; q,k,v = Wq/Wk/Wv x;
 * per-head RMSNorm of q and k (q_norm, k_norm), then NEOX RoPE at position pos
 * (pairs (i, i + head_dim/2)); k, v rounded to fp16 into cache slot pos; GQA
 * attention of q head h over kv head h / (n_heads/n_kv_heads), positions
 * 0..pos, scale 1/sqrt(head_dim); h += Wo attn; h += MoE(RMSNorm(h)*ffn_norm).
 * Sources: aprender issue "Qwen3 GPU inference produces garbage output" (Fix
 * Applied), aprender PR "apply per-head Q/K RMSNorm in forward_qwen3_moe" (The
 * fix), SharpInference issue "Forward-pass divergence on Qwen3-Coder 30B-A3B"
 * (NEOX RoPE).  ids_out (nullable): int32 [n_layers][k] selected experts.
 * Requires the attention geometry in the config; 0 <= pos < max_ctx. */
qmoe_status qmoe_decode_step(qmoe_ctx* ctx, const qmoe_layer_weights* layers, int n_layers,
                             int pos, float* hidden, int32_t* ids_out);

/* Batched prefill: n_tokens tokens at positions pos0 .. pos0+n_tokens-1 through
 * n_layers qwen3moe decoder layers, in place on hidden (F32 [n_tokens][H],
 * device, 16-byte aligned).  Per layer it computes, for every token t, what
 * qmoe_decode_step computes for one token at position pos0 + t, with causal
 * attention: token t attends to the cache positions 0 .. pos0-1 as stored and
 * to the batch's tokens 0 .. t.  Within a layer a token's K and V depend only
 * on its own input, so this equals n_tokens decode steps in order (the
 * token-by-token prefill of the aprender issue "qwen3moe ... has NO working
 * CUDA path", later gap list, "Prefill is token-by-token", which names the
 * batched form as the fix).  Differences from the decode step: the Q/K/V and O
 * projections run as tensor-core GEMMs on fp16 rows of the normalised input and
 * of the attention output (fp32 accumulation), and for n_tokens > 8 the MoE is
 * the tensor-core grouped-GEMM path of qmoe_forward_ex (fp16 operands).
 *  layers   : n_layers qmoe_layer_weights, as for qmoe_decode_step; the cache
 *             slots pos0 .. pos0+n_tokens-1 of every layer are written (fp16),
 *             the other slots are only read.
 *  ids_out  : nullable, int32 [n_layers][n_tokens][k] selected experts.
 * Requires the attention geometry in the config with at most 8 q heads per kv
 * head and n_heads*head_dim, n_kv_heads*head_dim multiples of 128; otherwise
 * QMOE_ERR_SHAPE.  1 <= n_tokens <= max_tokens, 0 <= pos0, pos0 + n_tokens <=
 * max_ctx (else QMOE_ERR_SHAPE).  The context holds a scratch of
 * about 56 KiB per max_tokens token at the Qwen3-30B-A3B shape for this call. */
qmoe_status qmoe_prefill(qmoe_ctx* ctx, const qmoe_layer_weights* layers, int n_layers,
                         int n_tokens, int pos0, float* hidden, int32_t* ids_out);

/* ------------------------------------------------------------------ paged 4-bit KV cache
 *
 * Several sequences share one pool of KV pages per layer, held in NVFP4 (the
 * format of qmoe_forward_nvfp4): E2M1 codes two per byte with the even element
 * in the low nibble, one E4M3 scale per 16 consecutive elements of a head, one
 * fp32 scale per kv head.  A position of a kv head takes head_dim * 9/16 bytes
 * for K and as much for V (144 B together at head_dim 128, against 512 B in the
 * fp16 cache of qmoe_decode_step).  One layer's cache:
 *   codes  [n_pages][n_kv_heads][page_size][head_dim/2]   bytes
 *   scales [n_pages][n_kv_heads][page_size][head_dim/16]  E4M3 codes, not NaN
 *   value (page, kv head, slot, d) = e2m1(code) * e4m3(scale[d/16]) * global[kv head]
 * A slot is page * page_size + offset (int64).  Position p of sequence s lives in
 * page block_table[s][p / page_size] at offset p % page_size.
 *
 * A serving step is qmoe_kv4_plan once, then per layer qmoe_kv4_append and
 * qmoe_kv4_attention (qmoe_step_kv4 runs whole decoder layers that way).  All
 * lengths, tables and slots stay on the device, so a step can be captured into a
 * graph and replayed while the lengths change.
 *
 * Conventions as above.  A qmoe_kv4 handle has its own stream, workspace, status
 * word and error text; a call runs on the device the handle was created on,
 * whichever device is current.  Calls that share a handle share its workspace:
 * they must be ordered (graphs captured from one handle must not run at the same
 * time).  Contents of device arrays are checked on the device: an index outside
 * its range is never followed, and sets the status word (QMOE_ERR_DEVICE_CHECK).
 * Waits between CTAs are bounded: one that runs out sets QMOE_ERR_TIMEOUT, the rows
 * it was for are not written, and the handle serves the next call. */
typedef enum {
    QMOE_F32 = 0, QMOE_F16 = 1, QMOE_BF16 = 2,
    QMOE_E4M3 = 3           /* only where an entry point names it */
} qmoe_dtype;

typedef struct qmoe_kv4 qmoe_kv4;

typedef struct {
    int n_heads;            /* q heads, 1..1024 */
    int n_kv_heads;         /* kv heads, divides n_heads */
    int head_dim;           /* 64, 128 or 256 */
    int page_size;          /* positions per page: 16, 32, 64, 128 or 256 */
    int n_pages;            /* pages of each layer's cache, 1..2^30 */
    int max_seqs;           /* largest n_seqs of a call, 1..4096 */
    int max_tokens;         /* largest n_tokens of a call, 1..2^20 */
    int max_pages_per_seq;  /* row length of the block table; times page_size at most 2^30 */
    void* stream;           /* cudaStream_t the work is enqueued on (NULL = legacy default) */
} qmoe_kv4_config;

/* One layer's cache (all device pointers; codes and scales 16-byte aligned). */
typedef struct {
    void* k_codes;
    void* k_scales;
    void* v_codes;
    void* v_scales;
    const float* k_global;  /* [n_kv_heads], finite; rows of a head whose global is not
                               positive are appended as zeros */
    const float* v_global;  /* [n_kv_heads], finite; attention's results lose bits where one
                               is smaller than 2^-80 (divided by the weights' sum it may
                               be subnormal) */
} qmoe_kv4_cache;

/* Create a handle on the current device and allocate its workspace (parts of
 * attention items that several CTAs share: 3 to 10 MB for decoding, 20 to 40 MB more
 * where a call may bring more than 16 rows of q, tokens times n_heads/n_kv_heads).
 * On failure qmoe_last_error(NULL) tells why. */
qmoe_status qmoe_kv4_create(const qmoe_kv4_config* cfg, qmoe_kv4** out);
void qmoe_kv4_destroy(qmoe_kv4* kv);
qmoe_status qmoe_kv4_set_stream(qmoe_kv4* kv, void* stream);
size_t qmoe_kv4_workspace_bytes(const qmoe_kv4_config* cfg);   /* 0 on bad config */

/* As qmoe_get_status and qmoe_last_error, for a handle. */
qmoe_status qmoe_kv4_get_status(qmoe_kv4* kv);
const char* qmoe_kv4_last_error(qmoe_kv4* kv);

/* Block tables and slot maps of one step, from the requests' lengths (one launch).
 *  seq_len     : int32 [n_seqs] positions each request has cached.
 *  new_len     : int32 [n_seqs] tokens that arrive in this step, 0 for none;
 *                negative: the request has finished and returns its pages.
 *  block_table : int32 [n_seqs][max_pages_per_seq], in/out.  Columns below
 *                ceil(seq_len/page_size) are read; the columns that the new tokens
 *                reach are written; every other entry is left as it was.
 *  free_pages  : int32 [n_pages], in/out, a stack whose first *n_free entries are
 *                the free pages.  The pages of finished requests are pushed in
 *                the order of requests and columns, then the pages that new tokens
 *                need are popped in that order.  Entries below the final height
 *                are as after those pushes and pops, those above unspecified.
 *  n_free      : int32 [1].
 *  cap_tokens  : entries of positions and slots, 1..max_tokens.
 * Outputs (device):
 *  seq_len_out : int32 [n_seqs] lengths after the step (0 for a finished request);
 *                may be seq_len.
 *  n_free_out  : int32 [1]; may be n_free.
 *  cu_tokens   : int32 [n_seqs+1], the new tokens of request s are the rows
 *                cu_tokens[s] .. cu_tokens[s+1]-1 of the step's batch.
 *  positions   : int32 [cap_tokens], slots: int64 [cap_tokens], of each row; -1 in
 *                the rows behind the last token.
 * A step that cannot be served changes nothing: cu_tokens is all zero, positions
 * and slots are -1, lengths, tables and the free list stay, and the status word
 * says why: QMOE_ERR_DEVICE_CHECK (a length or n_free out of range, more pages
 * free than exist), QMOE_ERR_SHAPE (more than cap_tokens new tokens, or a request
 * longer than its table row), QMOE_ERR_NO_MEMORY (too few free pages).
 * Page ids are not what a step is refused for: one outside 0..n_pages-1 that the step
 * pushes, pops or gives a token a slot in stays as it is in table and stack, its
 * tokens have slot -1, and the status is QMOE_ERR_DEVICE_CHECK. */
qmoe_status qmoe_kv4_plan(qmoe_kv4* kv, int n_seqs, const int32_t* seq_len, const int32_t* new_len,
                          int32_t* block_table, int32_t* free_pages, const int32_t* n_free,
                          int cap_tokens, int32_t* seq_len_out, int32_t* n_free_out,
                          int32_t* cu_tokens, int32_t* positions, int64_t* slots);

/* Quantise n_tokens K and V rows into their slots (one launch).  Row t of kv head h
 * starts at k + t*k_stride + h*head_dim (elements of dtype; 0: n_kv_heads*head_dim),
 * so rows may be read in place from side-by-side Q/K/V rows.  Per 16 elements, in
 * fp32 (as qmoe_nvfp4_quantize, the global scale being given):
 *   s = E4M3 nearest to max|x| / (6 * global), ties to even, saturating at 448;
 *   d = e4m3(s) * global;  code = E2M1 nearest to x / d, ties to even, saturating
 *   at 6; all zero where d = 0.
 *  slots       : int64 [n_tokens]; a row whose slot is negative goes nowhere.  Slots
 *                that occur twice end up with an unspecified mixture of their rows;
 *                a slot past the cache is skipped (QMOE_ERR_DEVICE_CHECK).
 *  k_hat, v_hat: F32 [n_tokens][n_kv_heads*head_dim] or NULL: the values the cache
 *                holds for each row (also for rows that go nowhere).
 * Row base addresses, strides in bytes, k_hat and v_hat 16-byte aligned.  Inputs
 * must be finite (the codes of a 16-element block with NaN or infinity are
 * unspecified; its scale is never NaN). */
qmoe_status qmoe_kv4_append(qmoe_kv4* kv, const qmoe_kv4_cache* cache, const void* k, const void* v,
                            qmoe_dtype dtype, int n_tokens, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, float* k_hat, float* v_hat);

/* Causal GQA attention of a ragged batch of tokens over the cache.
 *  q           : n_tokens rows of n_heads*head_dim elements of q_t, q_stride elements
 *                apart (0: contiguous).  Rows cu_tokens[s] .. cu_tokens[s+1]-1 are the
 *                last cu_tokens[s+1]-cu_tokens[s] positions of sequence s; row i of the
 *                N rows of a sequence of seq_len[s] positions sees the positions
 *                0 .. seq_len[s]-N+i (their K and V appended before this call).
 *  max_new     : no sequence has more new tokens than this (1..n_tokens).
 *  seq_len     : int32 [n_seqs] lengths with the new tokens (qmoe_kv4_plan's output).
 *  scale       : softmax scale, finite, e.g. 1/sqrt(head_dim).
 *  out         : rows of n_heads*head_dim elements of out_t, out_stride apart (0:
 *                contiguous); sum over visible p of softmax(scale * q.k_p) v_p.
 *  lse         : F32 [n_tokens][n_heads] or NULL: log of the sum of exp(scale * q.k_p).
 * A row that sees no position is 0 with lse -inf.  Rows behind cu_tokens[n_seqs] are
 * left as they were.  q head h reads kv head h / (n_heads/n_kv_heads).  Products
 * have fp32 accumulators and the running maximum and sum are fp32; F32 rows and
 * their softmax weights enter the tensor cores as two fp16 terms each (22 bits), F16
 * and BF16 rows and their weights as one (11 bits, whatever out_t is; K and V are
 * exact in fp16).  Scores have to be in fp32's range.  A sequence whose offsets, length or new tokens are out of range
 * (negative, past the table row, n_tokens or max_new) is skipped, a position whose
 * page id is out of range counts as not visible, and offsets that descend anywhere
 * leave all rows as they were; each sets QMOE_ERR_DEVICE_CHECK.  Row addresses,
 * strides in bytes and out 16-byte aligned; out must not overlap q. */
qmoe_status qmoe_kv4_attention(qmoe_kv4* kv, const qmoe_kv4_cache* cache, const void* q,
                               qmoe_dtype q_t, int64_t q_stride, int n_seqs, int n_tokens,
                               int max_new, const int32_t* cu_tokens, const int32_t* seq_len,
                               const int32_t* block_table, float scale, void* out,
                               qmoe_dtype out_t, int64_t out_stride, float* lse);

/* One serving step of a ragged batch through n_layers qwen3moe decoder layers over
 * paged 4-bit caches, in place on hidden (F32 [n_tokens][H], device): the layer of
 * qmoe_prefill for n_tokens tokens of n_seqs sequences, each at its own position,
 * with its K and V rows appended (qmoe_kv4_append) and attended to
 * (qmoe_kv4_attention, q rows and output as fp16) in caches[l] instead of the
 * layers' own fp16 caches (k_cache and v_cache of the layers are not used and may
 * be NULL).  The caches' globals are the caller's choice, made before the rows are
 * known: what is larger than 2688 globals is appended as that.  Decoding, draft tokens and prompt chunks may share a call.
 *  kv        : handle with the context's n_heads, n_kv_heads and head_dim, on its
 *              device (where the call runs, whichever is current) and stream.
 *  cu_tokens, seq_len, block_table, positions, slots : of the step, as
 *              qmoe_kv4_plan gives them; max_new as for qmoe_kv4_attention.
 *  ids_out   : nullable, int32 [n_layers][n_tokens][k] selected experts.
 * Rows that qmoe_kv4_attention would not write (behind cu_tokens[n_seqs] in a padded
 * batch, of a sequence that is skipped) are left as they were, their ids unspecified;
 * their K and V go where slots says.  Requires the attention geometry in the config and the shapes of
 * qmoe_prefill; max_ctx does not bound the positions.  Device-side findings are in
 * the status words of both the context and the handle. */
qmoe_status qmoe_step_kv4(qmoe_ctx* ctx, qmoe_kv4* kv, const qmoe_layer_weights* layers,
                          const qmoe_kv4_cache* caches, int n_layers, int n_seqs, int n_tokens,
                          int max_new, const int32_t* cu_tokens, const int32_t* seq_len,
                          const int32_t* block_table, const int32_t* positions,
                          const int64_t* slots, float* hidden, int32_t* ids_out);

/* ------------------------------------------------------------------ the 8-bit path's rows
 *
 * What a decoder layer over FP8 weights needs around qmoe_forward_fp8 and the paged
 * cache: the norms, 8-bit activations, dense products on them, rotary positions and
 * the append that rotates.  In the order of a layer:
 *   qmoe_rmsnorm (residual added, 8 bits out), qmoe_linear_fp8 (Q/K/V),
 *   qmoe_kv4_append_rope, qmoe_kv4_attention, qmoe_fp8_quantize, qmoe_linear_fp8 (O,
 *   residual added), qmoe_rmsnorm, qmoe_forward_fp8.
 *
 * 8-bit rows: E4M3 codes [rows][cols], contiguous, and one F32 scale per 128
 * consecutive elements of a row [rows][ceil(cols/128)]; value = e4m3(code) * scale.
 * Made in fp32: scale = max|y| of the block / 448; code = E4M3 nearest to y / scale,
 * ties to even, saturating; zero where the scale is 0 (max|y| / 448 may be too small
 * for fp32).  A NaN has the NaN code and does not count for the maximum; in a block
 * with an infinity the scale is infinite, the infinity's code NaN, the finite ones' 0.
 *
 * Conventions as above.  The calls on a qmoe_ctx use its stream and run on its device,
 * whichever is current; none has a workspace, so max_tokens does not bound them.
 * Strides are in elements of the rows' type, 0 for contiguous rows; row base
 * addresses and strides in bytes are multiples of 16.  Unless said otherwise outputs
 * must not overlap inputs. */

/* h = x (+ residual); y = h / sqrt(mean(h^2) + eps) (* weight), for n_rows rows of dim
 * elements (one launch).  The sum, its mean square and the quotient are fp32, from h
 * before it is rounded to res_t; squares have to be in fp32's range.
 *  x        : rows of x_t (F32, F16, BF16), x_stride apart.
 *  residual : rows of res_t, res_stride apart, or NULL (then res_t and res_stride are
 *             not used).
 *  sum      : rows of res_t, res_stride apart, h itself, or NULL; may be the residual, or
 *             x of that type and stride.  Only with a residual.
 *  weight   : F32 [dim], 16-byte aligned, or NULL (1).
 *  eps      : positive, finite.
 *  n_rows 1..2^24, dim a multiple of 16 up to 32768.
 *  y        : rows of y_t, y_stride apart (F32, F16, BF16; may be x of that type and
 *             stride), or 8-bit rows (QMOE_E4M3; y_stride 0 or dim).
 *  y_scale  : F32 [n_rows][ceil(dim/128)] for 8-bit rows, else NULL. */
qmoe_status qmoe_rmsnorm(qmoe_ctx* ctx, const void* x, qmoe_dtype x_t, int64_t x_stride,
                         const void* residual, qmoe_dtype res_t, int64_t res_stride, void* sum,
                         const float* weight, float eps, int n_rows, int dim, void* y,
                         qmoe_dtype y_t, int64_t y_stride, float* y_scale);

/* n_rows rows of cols elements of x_t as 8-bit rows (one launch).  cols a multiple of
 * 16 up to 32768, n_rows 1..2^24. */
qmoe_status qmoe_fp8_quantize(qmoe_ctx* ctx, const void* x, qmoe_dtype x_t, int64_t x_stride,
                              int n_rows, int cols, void* codes, float* scale);

typedef enum {
    QMOE_ACT_NONE = 0,
    QMOE_ACT_RELU = 1,
    QMOE_ACT_SILU = 2,     /* z / (1 + exp(-z)) */
    QMOE_ACT_GELU = 3      /* z * (1 + erf(z / sqrt 2)) / 2, to 2e-7 |z| */
} qmoe_act;

/* out = act(x W^T + bias) + residual (one launch).
 *  x_codes, x_scale : 8-bit rows [n_tokens][in_features] (codes 16-byte aligned).
 *  w_codes : E4M3 [out_features][in_features], 16-byte aligned; w_scale: F32, one per
 *            128 x 128 block, [ceil(out_features/128)][ceil(in_features/128)] (the weights
 *            of qmoe_forward_fp8, with blocks cut at the edges).
 *  bias    : F32 [out_features] or NULL.
 *  residual: rows of out_t, res_stride apart, or NULL; may be out with the same stride.
 *  out     : rows of out_t (F32, F16, BF16), out_stride apart, at least out_features.
 *  in_features a multiple of 16 up to 2^20, n_tokens 1..2^24, out_features 1..2^24.
 * Products of codes are accumulated in fp32 by blocks of 128, each block's sum scaled
 * and added in fp32, in an order that the sizes and the GPU decide.  The product of a
 * token's and a block's scale has to be in fp32's range.  Only the out_features first
 * elements of a row of out are written.  A bounded wait that runs out sets
 * QMOE_ERR_TIMEOUT, the call's results are then unspecified. */
qmoe_status qmoe_linear_fp8(qmoe_ctx* ctx, const void* x_codes, const float* x_scale, int n_tokens,
                            int in_features, const void* w_codes, const float* w_scale,
                            int out_features, const float* bias, qmoe_act act, const void* residual,
                            int64_t res_stride, void* out, qmoe_dtype out_t, int64_t out_stride);

/* Rotary positions.  Pair j of a head (j < rot_dim/2) is turned by the angle p * f_j at
 * position p; elements from rot_dim on stay as they are.
 *   pairs: (j, j + rot_dim/2) in QMOE_ROPE_HALF, (2j, 2j + 1) in QMOE_ROPE_INTERLEAVED
 *   f_j = base^(-2j/rot_dim), then
 *     QMOE_ROPE_LINEAR: f_j / factor
 *     QMOE_ROPE_PARTS : f_j (1 - r_j) + f_j / factor r_j, where r_j rises from 0 at pair
 *       max(0, floor(d(beta_fast))) to 1 at min(rot_dim - 1, ceil(d(beta_slow))), at least
 *       0.001 pairs further on, d(t) = rot_dim ln(orig_ctx / (2 pi t)) / (2 ln base) being the
 *       pair that turns t times in orig_ctx positions (YaRN, Peng et al. 2023)
 * mscale multiplies cosines and sines; 0 stands for 0.1 ln(factor) + 1 with
 * QMOE_ROPE_PARTS (factor > 1), else 1. */
typedef enum { QMOE_ROPE_HALF = 0, QMOE_ROPE_INTERLEAVED = 1 } qmoe_rope_layout;
typedef enum { QMOE_ROPE_PLAIN = 0, QMOE_ROPE_LINEAR = 1, QMOE_ROPE_PARTS = 2 } qmoe_rope_scaling;
typedef struct {
    int layout;             /* qmoe_rope_layout */
    int rot_dim;            /* elements of a head that are turned, a multiple of 16, 16..256 */
    int scaling;            /* qmoe_rope_scaling */
    int n_pos;              /* positions of the table, 1..2^24 */
    double base;            /* > 1 */
    double factor;          /* LINEAR, PARTS: > 0 */
    double orig_ctx;        /* PARTS: > 0 */
    double beta_fast;       /* PARTS: > beta_slow */
    double beta_slow;       /* PARTS: > 0 */
    double mscale;          /* >= 0 */
    float* table;           /* F32 [n_pos][2][rot_dim/2], cosines and sines, 16-byte aligned */
} qmoe_rope_config;

/* Fill rope->table (angles, cosines and sines in 64 bits, rounded once): made once, and
 * kept by the caller for the calls below. */
qmoe_status qmoe_rope_table(qmoe_ctx* ctx, const qmoe_rope_config* rope);

/* Rows of n_heads heads, each normalised on demand and turned (one launch):
 *   n = x / sqrt(mean(x^2) + eps) * norm   over a head, where norm is not NULL
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * every product, sum and quotient fp32, rounded once (no fused multiply-add); the mean
 * square of a head in more bits, its inverse root rounded to fp32 (to the nearest, or the
 * other where the root lies within 2^-34 of the border between two: one head in a million).
 *  rope      : layout, rot_dim (at most head_dim), n_pos and table are used.
 *  x, out    : n_tokens rows of n_heads*head_dim elements of x_t, x_stride and out_stride
 *              apart; out may be x with the same stride.
 *  head_dim  : 64, 128 or 256.  n_tokens 1..2^20, n_heads 1..1024.
 *  positions : int32 [n_tokens].  A row of a negative position (padding) is left as
 *              it was in out, one of a position past the table too, and that sets
 *              QMOE_ERR_DEVICE_CHECK.
 *  norm      : F32 [head_dim], 16-byte aligned, or NULL (then eps is not used). */
qmoe_status qmoe_rope(qmoe_ctx* ctx, const qmoe_rope_config* rope, const void* x, qmoe_dtype x_t,
                      int64_t x_stride, int n_tokens, int n_heads, int head_dim,
                      const int32_t* positions, const float* norm, float eps, void* out,
                      int64_t out_stride);

/* qmoe_kv4_append with qmoe_rope before it (one launch): the K rows are normalised (k_norm)
 * and turned as there and appended with the V rows, and the q rows are turned (q_norm)
 * into q_out; sizes and heads are the handle's.
 *  rope     : rot_dim a multiple of 32 (at most head_dim).
 *  q, q_out : rows of n_heads*head_dim elements of dtype, q_stride and q_out_stride apart;
 *             q_out may be q with the same stride.  Both NULL: only K and V.
 *  k, v     : rows of n_kv_heads*head_dim elements of dtype, as for qmoe_kv4_append.
 *  positions: int32 [n_tokens], as for qmoe_rope; K and V of a row without a position go
 *             nowhere, and its q_out, k_hat and v_hat are left as they were.
 *  slots, k_hat, v_hat : as for qmoe_kv4_append (k_hat: the turned rows as the cache
 *             holds them).
 *  q_norm, k_norm : F32 [head_dim], 16-byte aligned, or NULL. */
qmoe_status qmoe_kv4_append_rope(qmoe_kv4* kv, const qmoe_kv4_cache* cache,
                                 const qmoe_rope_config* rope, const void* q, const void* k,
                                 const void* v, qmoe_dtype dtype, int n_tokens, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const int32_t* positions,
                                 const int64_t* slots, const float* q_norm, const float* k_norm,
                                 float eps, void* q_out, int64_t q_out_stride, float* k_hat,
                                 float* v_hat);

/* Allocation-free variant of qmoe_forward for decode-sized calls.  The pages
 * have no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory: processes whose device memory is owned by their own
 * pool (a host framework's allocator, a plugin inside such a process), or
 * latency-critical loops that must not run a cudaMalloc, with its implicit
 * device synchronisation, after start-up.  It needs no context and allocates
 * nothing: its scratch (the tagged router logits, SwiGLU activations and down
 * outputs that the fused decode kernel passes between its CTAs, the "x staged"
 * marks, two control words and a status word) is one fixed device array inside
 * the library of 2 MiB + 256 B, which every GPU that loads the library holds
 * until the process exits.
 *  - Computes the same as qmoe_forward (hidden_out = hidden_in + MoE(hidden_in))
 *    with the same argument meaning, layout and alignment rules, on `stream`
 *    (a cudaStream_t; NULL = legacy default stream).
 *  - Served shapes: those of the fused single-kernel decode path (n_tokens
 *    <= 8, gate/up Q4_K, hidden in {256, 2048}, ffn in {256, 768}; see
 *    qmoe_fused_decode_available) whose buffers fit the array:
 *    8 * (n_tokens*n_experts + n_tokens*top_k*(ffn + hidden) + number of SMs)
 *    + 4 * top_k*ffn, each of the five parts rounded up to 256 B, at most 2 MiB.  At the
 *    Qwen3-30B-A3B shape that is every n_tokens <= 8 at top_k 8.  Anything
 *    else returns QMOE_ERR_SHAPE and enqueues nothing.
 *  - The first call on a device looks up the scratch's device address
 *    (cudaGetSymbolAddress) and sets the kernel's shared-memory limit; make that
 *    first call before any stream capture.
 *  - All calls share the one scratch array and it keeps the last call's
 *    contents.  Its control words carry over from call to call (they count
 *    launches, so values left by an earlier call are never mistaken for this
 *    call's); the status word is cleared at the start of every call.  Calls
 *    whose execution overlaps on the GPU (other streams, other host threads)
 *    race on it and give wrong results: order them.
 *  - Returns launch / argument errors only; the device-side status of the call
 *    (a bounded wait that ran out) is read with qmoe_noalloc_status. */
qmoe_status qmoe_forward_noalloc(const float* hidden_in, const float* router_w,
                                 const void* gate_exps, const void* up_exps,
                                 const void* down_exps, qmoe_qtype gate_t, qmoe_qtype up_t,
                                 qmoe_qtype down_t, int hidden, int n_experts, int top_k,
                                 int ffn, int norm_topk_prob, int n_tokens, float* hidden_out,
                                 void* stream);

/* Device-side status of the last qmoe_forward_noalloc call on the current
 * device: synchronises `stream` (the stream that call used), reads the status
 * word of the shared scratch and clears it.  QMOE_OK, or QMOE_ERR_TIMEOUT /
 * QMOE_ERR_DEVICE_CHECK as for qmoe_get_status; QMOE_ERR_CUDA if the device
 * was never set up by a call. */
qmoe_status qmoe_noalloc_status(void* stream);

/* Synchronise the stream and read the device status word (bounded-wait
 * timeouts, device index checks).  A non-OK status is sticky until read:
 * reading it clears it. */
qmoe_status qmoe_get_status(qmoe_ctx* ctx);

/* One-line description of the last error on this context ("" if none).  The
 * string is owned by the context and valid until the next call on it.  With
 * ctx = NULL: why the last qmoe_create on this thread failed (for
 * QMOE_ERR_NO_MEMORY the bytes the workspace needs and the bytes free). */
const char* qmoe_last_error(qmoe_ctx* ctx);

/* Test hooks (no counterpart on the pages).
 * qmoe_debug_stall_next: the next fused decode launch on this context (a
 *   qmoe_forward / qmoe_forward_ex of n_tokens <= 8 at a fused shape) waits for
 *   router logits carrying a launch tag that no CTA writes, gives up after
 *   wait_ns, records QMOE_ERR_TIMEOUT in the status word and exits without
 *   computing (its outputs are left unwritten).  Later launches are normal:
 *   this is how a test shows that a timed-out launch leaves the context usable.
 * qmoe_kv4_debug_stall_next: in the next qmoe_kv4_attention or qmoe_step_kv4 (its
 *   first layer) on this handle the CTAs that share an item of a prompt chunk hand
 *   their parts over wait_ns late (1..10^9); past 200 ms the CTA that joins them
 *   gives up: QMOE_ERR_TIMEOUT, the item's rows left unwritten.
 * qmoe_debug_stall_linear_next: in the next qmoe_linear_fp8 on this context, where pairs of
 *   CTAs take it and it has F32 rows and no activation, one CTA gets its scales wait_ns late
 *   (1..10^9); past 200 ms its pair gives up: QMOE_ERR_TIMEOUT, the call's results are unspecified.
 * qmoe_debug_fail_alloc: the next n workspace allocations of qmoe_create and
 *   qmoe_kv4_create, in any thread, fail as if the device were out of memory
 *   (QMOE_ERR_NO_MEMORY).
 * qmoe_debug_linear_choice: which kernel qmoe_linear_fp8 takes for these sizes on a GPU of
 *   num_sms multiprocessors: the features of a tile of a pair of CTAs (128 or 256) and how
 *   many pairs share its k (1 to 4), or tile 0 for the kernel of few tokens.  Pure host
 *   query; a test of a kernel asks it whether its sizes still go there. */
qmoe_status qmoe_debug_stall_next(qmoe_ctx* ctx, uint64_t wait_ns);
qmoe_status qmoe_kv4_debug_stall_next(qmoe_kv4* kv, uint64_t wait_ns);
qmoe_status qmoe_debug_stall_linear_next(qmoe_ctx* ctx, uint64_t wait_ns);
void qmoe_debug_fail_alloc(int n);
qmoe_status qmoe_debug_linear_choice(int num_sms, int n_tokens, int in_features, int out_features,
                                     int* tile, int* parts);

/* Bytes of workspace a context with this config allocates (0 on bad config). */
size_t qmoe_workspace_bytes(const qmoe_config* cfg);

/* 1 when qmoe_forward / qmoe_forward_ex on this context would run a layer of
 * n_tokens tokens with these expert qtypes as the single fused decode kernel
 * (one launch: router, top-k, gate/up, SwiGLU, down and combine), 0 when it
 * would take the multi-kernel path (tensor-core prefill or the SIMT path).
 * Pure host query; no device work. */
int qmoe_fused_decode_available(const qmoe_ctx* ctx, int n_tokens, qmoe_qtype gate_t,
                                qmoe_qtype up_t, qmoe_qtype down_t);

/* Byte stride between consecutive experts of a 3-D expert tensor whose
 * matrices have `rows` outputs and `cols` inputs (0 on bad arguments). */
size_t qmoe_expert_stride(qmoe_qtype qtype, int rows, int cols);

#ifdef __cplusplus
}
#endif

#endif /* QMOE_H */
