/*
 * bloom.h -- C ABI of the GB300 (sm_103a) BLOOM decoder engine.
 *
 * One job: KV-cached greedy token generation through a BLOOM-architecture
 * decoder stack on one GPU.  A generation is one prefill of the padded prompts
 * followed by one decode step per new token, the argmax token fed back in
 * ("Incredibly Fast BLOOM Inference with DeepSpeed and Accelerate", Benchmark
 * Environment: greedy, do_sample=False, KV cache enabled; per-token cost =
 * wall time / (batch x tokens)).
 *
 * The block (BLOOM as ported to transformers, "Optimization story: Bloom
 * inference", Porting to transformers):
 *   x = LN_emb(E[tok]);  per layer:  a = LN1(x); qkv = Wqkv a + bqkv;
 *   ALiBi attention with masked keys excluded and a float32 softmax
 *   ("Hugging Face BLOOM Inference Optimization", Custom CUDA Kernels);
 *   x += Wo o + bo;  x += Wdown gelu_tanh(Wup LN2(x) + bup) + bdown
 *   ("Kernel Fusion with torch.jit.script" for the GeLU);
 *   logits = E LN_f(x) (tied head); next = argmax, lowest index on ties.
 *
 * Conventions (all entry points):
 *  - Every tensor pointer is a DEVICE pointer owned by the caller unless the
 *    argument says "host".  The library borrows weights for the model's life.
 *  - Weights use the nn.Linear layout [out][in], row-major, bf16 (IEEE
 *    binary16-brain) or int8 with one bf16 scale per output row (W = q * s).
 *    Row pointers of every matrix must be 16-byte aligned (in % 8 == 0 for
 *    bf16, in % 16 == 0 for int8, base 16-byte aligned).
 *  - Fused QKV rows are head-interleaved: row (3*j + c)*d + e holds head j,
 *    c = 0 (query) / 1 (key) / 2 (value), element e, d = hidden / n_head.
 *  - Calls are asynchronous on the given CUDA stream (a cudaStream_t; NULL =
 *    the legacy default stream) and return a status validated on the host
 *    before anything is launched.  A kernel that meets a bad value (a token
 *    id >= vocab, a slot beyond the cache) records it in a device flag that
 *    bloom_check_device() reports; kernels never trap.
 *  - A model is not thread-safe; calls on one model must be issued in order
 *    on one stream.  Models are independent of one another.
 */
#ifndef BLOOM_H
#define BLOOM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BLOOM_OK = 0,
    BLOOM_E_INVALID = 1,      /* null / misaligned pointer, bad size or value */
    BLOOM_E_UNSUPPORTED = 2,  /* shape the kernels do not implement (see bloom_create) */
    BLOOM_E_OOM = 3,          /* device workspace allocation failed */
    BLOOM_E_CAPACITY = 4,     /* batch above the cache's, or cache full */
    BLOOM_E_CUDA = 5,         /* a CUDA runtime call failed; see bloom_last_error() */
    BLOOM_E_DEVICE_FLAG = 6   /* a kernel recorded a bad value (bloom_check_device) */
} bloom_status;

enum { BLOOM_WEIGHT_BF16 = 0, BLOOM_WEIGHT_INT8 = 1 };

/* flags */
enum {
    BLOOM_FLAG_NO_GRAPH = 1,  /* launch decode steps one kernel at a time (debug, profiling) */
    BLOOM_FLAG_NO_PDL = 2,    /* launch without programmatic dependent launch (each kernel
                                 waits for the previous one to finish before it starts) */
    BLOOM_FLAG_NO_LN_FUSION = 4, /* run every LayerNorm as its own kernel instead of inside
                                    the decode linear kernel that consumes it */
    BLOOM_FLAG_NO_TC_GEMM = 8    /* every linear on the weight-streaming kernel instead of the
                                    tensor-core (tcgen05) kernels: the prefill GEMM (>= 128
                                    tokens), the decode LM head (>= 3 sequences) and the decode
                                    block linears (bf16: every batch size where each block matrix
                                    is at most one wave of 128-row tiles, else >= 3 sequences;
                                    int8: 3..128 sequences) */
};

typedef struct {
    int32_t n_layer;
    int32_t hidden;        /* h; multiple of 256 */
    int32_t n_head;        /* n; head_dim d = h / n must be 64 or 128 */
    int32_t ffn;           /* F (4h in BLOOM); multiple of 256 */
    int32_t vocab;         /* V; the tied embedding has V rows */
    float   ln_eps;        /* LayerNorm epsilon (1e-5 in BLOOM) */
    int32_t weight_dtype;  /* BLOOM_WEIGHT_BF16 or BLOOM_WEIGHT_INT8 (block linears only;
                              the embedding / LM head is always bf16) */
    int32_t max_batch;     /* largest batch of any call */
    int32_t max_tokens;    /* largest B*T of any prefill (sizes the activation workspace) */
    int32_t max_seq;       /* largest cache length (prompt + generated) of any call */
    int32_t flags;         /* BLOOM_FLAG_* */
    int32_t wait_us;       /* bound of every wait of the tensor-core kernels in microseconds,
                              0 = about two seconds.  A wait that expires makes its launch give
                              up (stores skipped, memory it holds freed once its own copies and
                              MMAs have landed) and sets flag 8 for bloom_check_device; the model
                              stays usable.  Waits for the kernel's own copies and MMAs in
                              flight keep the default bound. */
} bloom_config;

/* One linear layer: bf16 weight, or int8 codes + bf16 row scales. */
typedef struct {
    const void *w;         /* bf16 [N][K] or int8 [N][K] */
    const void *scale;     /* bf16 [N] for int8, else NULL */
    const void *bias;      /* bf16 [N] or NULL (zero bias) */
} bloom_linear;

typedef struct {
    const void *ln1_g, *ln1_b;     /* bf16 [h] */
    bloom_linear qkv;              /* [3h][h] */
    bloom_linear o;                /* [h][h] */
    const void *ln2_g, *ln2_b;     /* bf16 [h] */
    bloom_linear up;               /* [F][h] */
    bloom_linear down;             /* [h][F] */
} bloom_layer_weights;

typedef struct {
    const void *word_emb;          /* bf16 [V][h]; also the tied LM head */
    const void *emb_ln_g, *emb_ln_b;
    const void *lnf_g, *lnf_b;
    const bloom_layer_weights *layers;   /* HOST array [n_layer] of device pointers */
} bloom_weights;

typedef struct bloom_model bloom_model;   /* opaque */

/* KV cache: one caller-owned device allocation of bloom_kv_bytes() bytes, one
 * row per sequence.  Layout (all regions 256-byte aligned): a 256-byte header,
 * int32 len[batch] (slots filled in each row), int32 active[batch] (1 = the row
 * takes part in decode steps), int32 next_pos[batch] (ALiBi position of each
 * row's next token), int32 pos[batch][max_seq] (position of each slot, -1 for a
 * pad slot), then K and V, each bf16 [n_layer][batch][n_head][max_seq][d].
 * The device copy is authoritative; the struct keeps a host mirror of the
 * per-row state, which the library updates on every call (the caller only
 * reads it).  Rows leave and join between decode steps (bloom_kv_retire,
 * bloom_kv_admit): "Hugging Face BLOOM Inference Optimization", Webserver
 * Architecture and Request Handling (dynamic batch extraction). */
#define BLOOM_MAX_BATCH 256
typedef struct {
    void   *buf;
    size_t  bytes;
    int32_t batch;
    int32_t max_seq;
    int32_t len;                              /* longest active row */
    int32_t row_len[BLOOM_MAX_BATCH];         /* slots filled, per row */
    uint8_t row_active[BLOOM_MAX_BATCH];      /* 1: the row decodes */
    void   *host_buf;                         /* K / V of layers >= offload_from (NULL: none) */
    size_t  host_bytes;
    int32_t offload_from;                     /* first layer kept in host_buf (n_layer: none) */
} bloom_kv;

/* Bytes a cache for `batch` sequences of `max_seq` slots needs (0 on bad args). */
size_t bloom_kv_bytes(const bloom_config *cfg, int32_t batch, int32_t max_seq);

/* Validate the config and weights, compute the ALiBi slopes once (largest
 * power of two m <= n heads: 2^(-8i/m), then every other term of the 2m
 * sequence), allocate the activation workspace, and pick launch shapes.
 * The current CUDA device is the model's device.  *out is NULL on failure.
 * For testing the error path, the environment variable BLOOM_INJECT_FAILURE
 * containing "workspace" makes the workspace allocation fail (BLOOM_E_OOM).
 * For testing that no kernel reads an activation before writing it, the
 * variable BLOOM_POISON_WORKSPACE fills the workspace with 0xff bytes (NaN in
 * bf16 and float32) instead of zeros, all but its tickets, argmax scratch and
 * flag word; results must not change. */
bloom_status bloom_create(const bloom_config *cfg, const bloom_weights *w, bloom_model **out);

/* Bind `buf` (device, >= bloom_kv_bytes bytes, 256-byte aligned) as an empty
 * cache and fill *kv: every row empty and idle, every slot a pad. */
bloom_status bloom_kv_init(bloom_model *m, bloom_kv *kv, void *buf, size_t bytes,
                           int32_t batch, int32_t max_seq, void *stream);

/* KV offload to host memory ("DeepSpeed Inference", IV.C.2 Offloading
 * Activations to CPU Memory: cached keys and values beyond what the GPU
 * should hold go to CPU memory, so that larger batches fit; IV.C.3 overlaps
 * the PCIe traffic with compute.  On GB300 the Grace memory is read and
 * written by the kernels themselves over NVLink-C2C, with no copies to
 * schedule): the K and V of layers [offload_from, n_layer) live in host_buf,
 * everything else in buf.  Sizes of both parts (offload_from = n_layer:
 * host_bytes = 0, device_bytes = bloom_kv_bytes).  BLOOM_E_INVALID on bad
 * arguments. */
bloom_status bloom_kv_bytes_offload(const bloom_config *cfg, int32_t batch, int32_t max_seq,
                                    int32_t offload_from, size_t *device_bytes,
                                    size_t *host_bytes);

/* bloom_kv_init with layers [offload_from, n_layer) in host_buf: page-locked
 * host memory (cudaHostAlloc / cudaMallocHost, 256-byte aligned) that the
 * device addresses with the same pointer -- checked, else BLOOM_E_INVALID.
 * The caller owns both buffers.  Decode and prefill kernels read and write the
 * offloaded layers' cache directly (zero-copy), at the host link's bandwidth. */
bloom_status bloom_kv_init_offload(bloom_model *m, bloom_kv *kv, void *buf, size_t bytes,
                                   void *host_buf, size_t host_bytes, int32_t batch,
                                   int32_t max_seq, int32_t offload_from, void *stream);

/* Prefill: run the B x T padded prompts (tokens int32 [B][T], mask uint8 [B][T],
 * 1 = token, 0 = pad; each row needs one token), write K,V of slots [0,T),
 * set slot positions (count of tokens before the slot), and emit the greedy
 * token of each row's last token slot to out_tokens int32 [B].  out_logits
 * (float [B][V]) may be NULL.  Requires B == kv->batch, T <= kv->max_seq,
 * B*T <= max_tokens.  Every row becomes active with length T. */
bloom_status bloom_prefill(bloom_model *m, bloom_kv *kv, const int32_t *tokens,
                           const uint8_t *mask, int32_t B, int32_t T, int32_t *out_tokens,
                           float *out_logits, void *stream);

/* One decode step: next_tokens int32 [B] of every active row go to the row's
 * next slot (row_len); out_tokens int32 [B] receives the greedy next token of
 * each active row and -1 for an idle one, and may alias next_tokens;
 * out_logits float [B][V] may be NULL (idle rows' logits are meaningless).
 * Unless BLOOM_FLAG_NO_GRAPH is set, the step is captured once per distinct
 * (kv, next_tokens, out_tokens, out_logits) into a CUDA graph and replayed; the
 * graph reads the rows' state on the device, so it stays valid across admit
 * and retire.  Each active row grows by one slot; BLOOM_E_CAPACITY if an active
 * row is full, BLOOM_E_INVALID if no row is active. */
bloom_status bloom_decode_step(bloom_model *m, bloom_kv *kv, const int32_t *next_tokens,
                               int32_t *out_tokens, float *out_logits, void *stream);

/* Per-member sampling (temperature + top-p) after the LM head: one decode step
 * (bloom_decode_step, logits into `logits`, float [B][V], device, required),
 * then each active row's next token drawn from its logits by bloom_op_sample
 * with its own temperature[b], top_p[b] and uniform number u[b] (device float
 * [B] each; the caller draws u, so the same inputs give the same tokens) into
 * out_tokens; idle rows get -1.  "Hugging Face BLOOM Inference
 * Optimization", Webserver Architecture and Request Handling: the custom
 * generation loop applies each batch member's own sampling parameters. */
bloom_status bloom_decode_step_sampled(bloom_model *m, bloom_kv *kv, const int32_t *next_tokens,
                                       int32_t *out_tokens, float *logits,
                                       const float *temperature, const float *top_p,
                                       const float *u, void *stream);

/* Dynamic batch: prefill n new prompts (tokens int32 [n][T], mask uint8 [n][T],
 * device) into the cache rows rows[i] (HOST int32 [n], distinct, < kv->batch),
 * leaving every other row untouched; those rows become active with length T
 * and take part in the next decode steps.  out_tokens int32 [n] (device)
 * receives each prompt's greedy token, out_logits float [n][V] may be NULL.
 * Requires n * T <= max_tokens. */
bloom_status bloom_kv_admit(bloom_model *m, bloom_kv *kv, const int32_t *rows, int32_t n,
                            const int32_t *tokens, const uint8_t *mask, int32_t T,
                            int32_t *out_tokens, float *out_logits, void *stream);

/* Dynamic batch: rows rows[i] (HOST int32 [n]) leave the batch: decode steps
 * no longer append to them (their out_tokens are -1) until an admit reuses
 * them. */
bloom_status bloom_kv_retire(bloom_model *m, bloom_kv *kv, const int32_t *rows, int32_t n,
                             void *stream);

/* Whole greedy generation with HOST buffers: copies tokens/mask (host int32 /
 * uint8 [B][T]) to the device, prefills, runs n_new - 1 decode steps feeding
 * each argmax back on the device, and copies the n_new tokens of every row to
 * out_host (host int32 [n_new][B]).  Synchronises the stream before returning
 * and reports a device flag as BLOOM_E_DEVICE_FLAG.  Requires T + n_new - 1
 * <= kv->max_seq. */
bloom_status bloom_generate(bloom_model *m, bloom_kv *kv, const int32_t *tokens_host,
                            const uint8_t *mask_host, int32_t B, int32_t T, int32_t n_new,
                            int32_t *out_host, void *stream);

/* Operations and kernels of a decode step, as bloom_decode_profile reports
 * them: code = op | (kernel << 8). */
enum {
    BLOOM_OP_EMBED = 0,       /* embedding gather + embedding LayerNorm */
    BLOOM_OP_LAYERNORM = 1,   /* LN1 / LN2 / ln_f as a kernel of its own */
    BLOOM_OP_QKV = 2,         /* fused QKV + bias + K/V append */
    BLOOM_OP_ATTN = 3,        /* ALiBi attention over the cache */
    BLOOM_OP_DENSE = 4,       /* attention output projection + bias + residual */
    BLOOM_OP_UP = 5,          /* MLP up projection + bias + GeLU */
    BLOOM_OP_DOWN = 6,        /* MLP down projection + bias + residual */
    BLOOM_OP_HEAD = 7         /* tied LM head + argmax */
};
enum {
    BLOOM_KERNEL_EMBED = 0,
    BLOOM_KERNEL_LAYERNORM = 1,
    BLOOM_KERNEL_STREAM = 2,          /* weight-streaming mma.sync linear */
    BLOOM_KERNEL_GEMV_TC = 3,         /* tensor-core (tcgen05) decode linear */
    BLOOM_KERNEL_GEMM_TC = 4,         /* tensor-core (tcgen05) prefill GEMM */
    BLOOM_KERNEL_ATTN = 5,            /* split-KV decode attention */
    BLOOM_KERNEL_ATTN_PREFILL = 6     /* prefill attention */
};

/* One decode step exactly as bloom_decode_step computes it (same kernels,
 * same results, kv->len advanced), but launched one kernel at a time, each
 * starting after the previous one has finished, with a CUDA event recorded
 * on `stream` after every launch; for measuring the share of each kernel in a
 * step.  Fills codes[i] (op | kernel << 8) and ms[i] (the launch's duration,
 * from the previous event) for the first min(cap, launches) launches, sets *n
 * to that count, and synchronises the stream.  codes, ms and n are HOST
 * pointers.  Not for use inside a stream capture. */
bloom_status bloom_decode_profile(bloom_model *m, bloom_kv *kv, const int32_t *next_tokens,
                                  int32_t *out_tokens, int32_t *codes, float *ms, int32_t cap,
                                  int32_t *n, void *stream);

/* Synchronise the stream, read and clear the device flag: BLOOM_OK or
 * BLOOM_E_DEVICE_FLAG (the flag's bits are in bloom_last_error()). */
bloom_status bloom_check_device(bloom_model *m, void *stream);

/* Free the workspace and graphs.  Caller-owned weights and caches are kept. */
bloom_status bloom_destroy(bloom_model *m);

/* Message of the last failing call on this thread ("" if none). */
const char *bloom_last_error(void);

/* Kernel launches one decode step of `batch` sequences issues (for launch
 * accounting): one per operation, less the LayerNorms fused into a linear. */
int32_t bloom_decode_launches(const bloom_model *m, int32_t batch);

/* ------------------------------------------------------------------------
 * Layer-level entry points.  They run one piece of the path on caller
 * buffers, with the same kernels the calls above use; tests use them to feed
 * each layer a reference input (teacher forcing) and to time one kernel.
 * ------------------------------------------------------------------------ */

/* The residual stream x of the layer-level calls is float32: it is the running
 * sum over layers and is kept unrounded; every other activation is bf16. */

/* One decoder layer of the decode step on x (float [kv->batch][h], in/out) for
 * the next token of every active row: it writes the layer's K,V at the row's
 * next slot and sets the slot position, but does not advance the rows. */
bloom_status bloom_layer_decode(bloom_model *m, bloom_kv *kv, int32_t layer, void *x,
                                void *stream);

/* Set the slot positions of a prompt (mask uint8 [B][T]) in the cache and
 * make every row active with length T, as the prefill does before its first
 * layer. */
bloom_status bloom_kv_set_prompt(bloom_model *m, bloom_kv *kv, const uint8_t *mask,
                                 int32_t B, int32_t T, void *stream);

/* One decoder layer of the prefill on x (float [B*T][h], in/out), writing K,V
 * of slots [0,T).  Needs bloom_kv_set_prompt first. */
bloom_status bloom_layer_prefill(bloom_model *m, bloom_kv *kv, int32_t layer, void *x,
                                 int32_t B, int32_t T, void *stream);

/* Final LayerNorm + tied LM head + argmax on x (float [B][h]): out_tokens int32
 * [B], out_logits float [B][V] or NULL. */
bloom_status bloom_head(bloom_model *m, const void *x, int32_t B, int32_t *out_tokens,
                        float *out_logits, void *stream);

/* Tied LM head + argmax alone (one kernel, the model's scratch) on rows that
 * are already normalised by ln_f: xn bf16 [B][h] -> out_tokens int32 [B],
 * out_logits float [B][V] or NULL.  Used to time the head in isolation. */
bloom_status bloom_lm_head(bloom_model *m, const void *xn, int32_t B, int32_t *out_tokens,
                           float *out_logits, void *stream);

/* Embedding gather + embedding LayerNorm: tokens int32 [n] -> x float [n][h]. */
bloom_status bloom_embed(bloom_model *m, const int32_t *tokens, int32_t n, void *x,
                         void *stream);

/* ------------------------------------------------------------------------
 * Operator entry points (no model needed), the kernels of the path on raw
 * buffers.  All bf16 tensors are row-major.
 * ------------------------------------------------------------------------ */

/* y[r] = LN(x[r]) * g + b over h features, float32 statistics, biased
 * variance, eps inside the square root; x, y bf16 [rows][h]; g, b bf16 [h]
 * (NULL: 1 and 0).  h % 8 == 0, h <= 16384. */
bloom_status bloom_op_layernorm(const void *x, const void *g, const void *b, int32_t rows,
                                int32_t h, float eps, void *y, void *stream);

enum {
    BLOOM_EPI_STORE = 0,   /* y = acc + bias */
    BLOOM_EPI_GELU = 1,    /* y = gelu_tanh(acc + bias) */
    BLOOM_EPI_RESID = 2    /* y = y + acc + bias (residual add in place) */
};

/* Weight-streaming linear layer y[M][N] (bf16) = epilogue(x[M][K] W^T + bias)
 * with float32 accumulation; W per bloom_linear.  K % 8 == 0 (bf16) or
 * K % 16 == 0 (int8). */
bloom_status bloom_op_linear(const bloom_linear *lin, int32_t int8, const void *x, int32_t M,
                             int32_t N, int32_t K, int32_t epilogue, void *y, void *stream);

/* The same linear layer on the tensor-core GEMM that prefill uses for batches
 * of >= 128 tokens ("DeepSpeed Inference", III.A and IV.C.1: prompt processing
 * is compute-bound): 128 x 256 output tiles, tcgen05.mma into TMEM, operands
 * moved by TMA.  bf16 weights only (lin->scale must be NULL); x and lin->w
 * 16-byte aligned; K % 8 == 0; any M >= 0 and N >= 1.  Same epilogues and
 * result layout as bloom_op_linear.  BLOOM_E_UNSUPPORTED if the driver cannot
 * describe the operands for TMA. */
bloom_status bloom_op_gemm(const bloom_linear *lin, const void *x, int32_t M, int32_t N,
                           int32_t K, int32_t epilogue, void *y, void *stream);

/* The same linear layer on the tensor-core decode kernel (the decode steps of
 * 3 or more sequences run their linears on it): W is the 128-row operand of
 * tcgen05.mma, the tokens its N operand, both moved by TMA, the accumulator in
 * TMEM; narrow matrices split K over a thread-block cluster whose partials are
 * summed in split order ("DeepSpeed Inference", III.A: small-batch cost is
 * reading W).  int8 = 0: bf16 weights, M <= 256, K % 8 == 0.  int8 = 1: int8
 * codes with bf16 row scales (lin->scale), widened exactly on the chip (to f16,
 * with the activations converted to f16, up to 32 rows; to bf16 above) and
 * scaled per row in the epilogue, M <= 128, K % 16 == 0 ("Incredibly Fast
 * BLOOM Inference...", Key observations: int8 halves the bytes read).  x and
 * lin->w 16-byte aligned.  Same epilogues and result layout as bloom_op_linear. */
bloom_status bloom_op_linear_tc(const bloom_linear *lin, int32_t int8, const void *x, int32_t M,
                                int32_t N, int32_t K, int32_t epilogue, void *y, void *stream);

/* Split-KV decode attention for one token per sequence.
 * q bf16 [B][n][d]; k_cache, v_cache bf16 [B][n][max_seq][d]; pos int32
 * [B][max_seq] (-1 = masked); keys are slots [0, len]; slopes float [n];
 * o bf16 [B][n*d].  d in {64, 128}.  `splits` key ranges per (b, head), 0 =
 * library choice.  q, k_cache, v_cache and o 16-byte aligned (BLOOM_E_INVALID
 * otherwise); K / V in device memory may be staged by bulk copies, K / V in
 * host memory are read directly. */
bloom_status bloom_op_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *pos, const float *slopes, int32_t B,
                                  int32_t n_head, int32_t d, int32_t max_seq, int32_t len,
                                  int32_t splits, void *o, void *stream);

/* Temperature + top-p sampling of B rows of float32 logits (row b at logits +
 * b * ld, ld >= V; device).  temperature, top_p, u: device float [B]; out_tokens:
 * device int32 [B].  Row b: p_i proportional to exp((z_i - max z) / temperature);
 * the nucleus is the shortest prefix of the tokens by probability (highest
 * first, equal logits in index order) whose mass reaches top_p; the token is
 * where the nucleus's cumulative mass in vocabulary order first exceeds u times
 * its mass.  temperature <= 0 or NaN: greedy argmax (lowest index on ties);
 * top_p >= 1 or NaN: every token with non-zero mass; top_p <= 0: the most
 * probable token; u < 0 or NaN counts as 0, u >= 1 takes the last nucleus
 * token.  Masses are 2^-40 fixed point of float32 exp, summed in 64-bit
 * integers: the result does not depend on summation order.  NaN logits, and
 * logits more than 27 temperature units below the maximum (mass below 2^-38
 * of the maximum's), take no part.  One cluster of 8 CTAs per row;
 * BLOOM_E_INVALID for null pointers, B outside 1..65535, V < 1 or ld < V. */
bloom_status bloom_op_sample(const float *logits, int32_t B, int32_t V, int64_t ld,
                             const float *temperature, const float *top_p, const float *u,
                             int32_t *out_tokens, void *stream);

/* Sampling with temperature, top-k, top-p and min-p of B rows of float32 logits (row
 * b at logits + b * ld, ld >= V), J draws a row.  temperature, top_p, min_p (float) and
 * top_k (int32): device arrays [B], or NULL for none (temperature 1); u: device
 * float [B][J]; out_tokens: device int32 [B][J].  Row b: p proportional to
 * exp((z - max z) / temperature); in the order of bloom_op_sample (probability,
 * highest first, equal logits by index) the kept tokens are the first top_k, of
 * those the shortest prefix that holds top_p of their mass, and of those the
 * ones with p >= min_p * max p.  Each draw takes the token where the kept mass,
 * summed in vocabulary order, first exceeds u times the whole of it.
 * temperature <= 0 or NaN, or top_p <= 0: the most probable token; a temperature
 * below 2^-126 counts as that.  Off: top_k <= 0,
 * top_p >= 1 or NaN, min_p <= 0 or NaN; min_p >= 1 keeps the tokens of the largest
 * logit.  u < 0 or NaN counts as 0, u >= 1 takes the last kept token with mass.
 * NaN and -inf logits take no part, nor do logits 40 or more binades of mass, or 2^128, below the
 * maximum; +inf logits share the whole mass.  Masses are 2^-40 fixed point, summed in
 * 64-bit integers: the result does not depend on the order of summation.  A row
 * where nothing takes part gives -1.  BLOOM_E_INVALID for null or misaligned
 * pointers, B outside 0..65535, V outside 1..2^22, ld < V, J outside 0..2^30 (B = 0 or
 * J = 0 does nothing). */
bloom_status bloom_op_sample_filtered(const float *logits, int32_t B, int32_t V, int64_t ld,
                                      const float *temperature, const int32_t *top_k,
                                      const float *top_p, const float *min_p, const float *u,
                                      int32_t J, int32_t *out_tokens, void *stream);

/* Log probabilities of given tokens, with entropy and top alternatives, of B rows
 * of float32 logits (row b at logits + b * ld, ld >= V; device), natural
 * logarithms of softmax(logits):
 *   logp[b][j]  of tokens[b][j] (device int32 [B][J]); a token -1 (no token: an
 *               idle row of a decode step) gets 0, any other value outside
 *               [0, V) NaN;
 *   entropy[b]  = -sum p log p, or NULL for none;
 *   top_ids[b][i], top_logp[b][i], i < top: the tokens with the highest logits,
 *               highest first, equal logits in index order.
 * As in bloom_op_sample, NaN logits take no part, nor do -inf ones: their
 * tokens' logp is -inf and they are never top alternatives; places left over
 * get id -1 and -inf.  A row where nothing takes part has entropy 0.  +inf
 * logits share the whole mass.  Sums are float32.  tokens / logp may be NULL
 * with J = 0, top_ids / top_logp with top = 0.  BLOOM_E_INVALID for null
 * pointers, B outside 0..65535, V < 1, ld < V, J < 0, top outside 0..32 (B = 0
 * does nothing). */
bloom_status bloom_op_logprobs(const float *logits, int32_t B, int32_t V, int64_t ld,
                               const int32_t *tokens, int32_t J, float *logp, float *entropy,
                               int32_t top, int32_t *top_ids, float *top_logp, void *stream);

/* ------------------------------------------------------------------------
 * 8-bit KV cache of one layer: codes with one float32 scale for every
 * BLOOM_KV8_BLOCK slots of a (row, head), K and V apart; value = code * scale.
 * Half the bytes of the bf16 cache for decode attention to read.
 * ------------------------------------------------------------------------ */
enum { BLOOM_KV8_INT8 = 0, BLOOM_KV8_E4M3 = 1 };
#define BLOOM_KV8_BLOCK 32

typedef struct {
    void *k, *v;               /* codes [batch][n_kv][max_seq][d], 16-byte aligned, device */
    float *k_scale, *v_scale;  /* [batch][n_kv][ceil(max_seq / BLOOM_KV8_BLOCK)], device */
    int32_t codes;             /* BLOOM_KV8_INT8: -127..127; BLOOM_KV8_E4M3: finite e4m3 */
    int32_t batch, n_kv, max_seq;
    int32_t d;                 /* 64 or 128 */
} bloom_kv8;

/* `flag` of the three calls below: a device int32 word, or NULL, that a kernel
 * ORs a bit of bloom_check_device into when it meets a bad value (2: a slot
 * beyond the cache; 8: a bounded wait of the attention expired: the outputs that
 * depend on what it waited for are NaN, the others right). */

/* Quantise new keys and values into the cache: token t of row b goes to slot
 * start[b] + t, t < count[b] (count NULL: T; clamped to 0..T).  k and v: bf16,
 * element (b, t, head, e) at b * stride[0] + t * stride[1] + head * stride[2] +
 * e, strides in elements, multiples of 8, k_stride and v_stride HOST arrays of
 * three (views of a fused QKV row, of [B][T][n][d] and of a bf16 cache's
 * [B][n][S][d] all fit; a stride may be 0); k and v 16-byte aligned.  start, count: device int32
 * [batch]; mask: device uint8 [batch][T] or NULL.
 *  - A block's scale is the smallest power of two, 2^-126 at least, with
 *    amax <= 127 * scale (int8) or 448 * scale (e4m3) over its tokens, 0 if all
 *    are 0; codes are value / scale rounded half to even.
 *  - A block that holds tokens already (slots below start[b]) keeps its scale
 *    unless the new tokens need a larger one: then the codes it holds are
 *    rounded again in the larger scale.  A block whose first slot is written
 *    starts afresh, whatever it held.  So a cache need not be cleared, provided
 *    each row is first written from a slot that is a multiple of 32.
 *  - mask 0 (a pad slot): the token is stored as zeros and not looked at.
 *  - start[b] < 0: row b is idle and left as it is, as are all blocks that the
 *    call writes no slot of.  Slots of a written block from the row's end (start[b] +
 *    count[b]) on keep their codes, but not their values: they count as free, and the
 *    block's scale may change without them.  A row that goes back writes again from
 *    there on.  Tokens beyond max_seq are dropped; flag 2 for those and for a row whose
 *    start lies beyond max_seq.
 *  - An infinity or NaN among a block's tokens makes its scale NaN: all of the
 *    block reads as NaN until it is started afresh.
 * The values must not overlap the cache.  T <= max_seq; T = 0 does nothing.
 * Calls that write one row, or read it, are issued in order (one stream, or
 * streams that wait for one another). */
bloom_status bloom_op_kv8_write(const bloom_kv8 *kv, const void *k, const int64_t *k_stride,
                                const void *v, const int64_t *v_stride, int32_t T,
                                const int32_t *start, const int32_t *count, const uint8_t *mask,
                                int32_t *flag, void *stream);

/* Read slots start[b] + t, t < T, back as bf16 values (rounded half to even;
 * exact for scales that bloom_op_kv8_write made) into k and v, addressed as in
 * bloom_op_kv8_write.  Tokens t >= count[b], of idle rows (start[b] < 0) and
 * beyond max_seq (flag 2) are written as 0.  The strides of the dimensions of
 * more than one element nest (BLOOM_E_INVALID otherwise): the smallest is at least d,
 * each next one at least what the smaller ones span; k, v and the cache must not overlap.
 * T <= max_seq; T = 0 does nothing. */
bloom_status bloom_op_kv8_read(const bloom_kv8 *kv, void *k, const int64_t *k_stride, void *v,
                               const int64_t *v_stride, int32_t T, const int32_t *start,
                               const int32_t *count, int32_t *flag, void *stream);

/* Decode attention over the cache for the last T tokens of every row (T = 1: a
 * decode step; up to 32: drafted tokens checked at once; their keys and values
 * are in the cache already).  q bf16 [batch][T][n_head][d]; query head j reads
 * key head j / (n_head / n_kv); pos int32 [batch][max_seq] as in
 * bloom_op_attn_decode (-1 = masked); slopes float [n_head], or NULL for no
 * position term; lens device int32 [batch]: slots filled, the new tokens
 * included.  Query t of row b sees slots [0, lens[b] - T + t]; one that sees
 * nothing (lens[b] <= 0: an idle row; all masked) gets 0.  lens[b] > max_seq
 * counts as max_seq (flag 2).  o bf16 [batch][T][n_head * d].  Masked slots and
 * slots from lens on are never looked at: they may hold anything.  A block with
 * a NaN scale makes every query that sees a slot of it NaN, in that head.
 * Scores, sums and outputs are float32 until the one rounding to bf16; a softmax
 * weight keeps 16 bits.  Its product with the V scale of its block counts down to
 * 2^-104 of the largest such product of the query (fewer bits, then 0, from there
 * on); elements of q below 2^-28 of the query's largest are off by up to 2^-39 of it.
 * batch * n_kv * max_seq is below 2^31 (BLOOM_E_UNSUPPORTED otherwise, as T > 32).
 * workspace: device scratch of bloom_op_attn_decode_kv8_workspace() bytes (0:
 * NULL will do), 16-byte aligned, contents immaterial; calls that may overlap on
 * the GPU (other streams, graphs that may run at once) need one each. */
bloom_status bloom_op_attn_decode_kv8(const bloom_kv8 *kv, const void *q, const int32_t *pos,
                                      const float *slopes, const int32_t *lens, int32_t T,
                                      int32_t n_head, void *o, void *workspace,
                                      size_t workspace_bytes, int32_t *flag, void *stream);

/* Bytes of that scratch; 0 also for arguments that the call refuses. */
size_t bloom_op_attn_decode_kv8_workspace(const bloom_kv8 *kv, int32_t T, int32_t n_head);

/* Bound of every wait of this thread's later bloom_op_attn_decode_kv8 calls, in
 * microseconds (0, the default: about two seconds).  A warp whose wait expires
 * stops there: it waits for its own copies in flight (at most three, about two
 * seconds each), sets flag 8, writes NaN for what is left of its work and ends.
 * BLOOM_E_INVALID below 0. */
bloom_status bloom_op_attn_decode_kv8_wait_us(int32_t wait_us);

/* ------------------------------------------------------------------------
 * 4-bit weights with group scales: value = code * scale, codes -7 .. 7, one
 * bf16 scale for every `group` neighbouring weights of a row of [n][k].  4.25
 * bits a weight at groups of 64 for a decode step to read.
 * ------------------------------------------------------------------------ */
typedef struct {
    void *tiles;           /* bloom_w4_bytes() bytes, 16-byte aligned, device: tiles of 16 rows x
                              256 columns, in the order that the linear layer reads them */
    int32_t n, k;          /* rows (outputs) and columns (inputs); k % 8 == 0 */
    int32_t group;         /* 32, 64 or 128 */
} bloom_w4;

/* Bytes of the tiles of [n][k] weights; 0 on bad sizes. */
size_t bloom_w4_bytes(int32_t n, int32_t k, int32_t group);

/* Quantise bf16 weights [n][k] (row i at w + i * ld elements; ld >= k, ld % 8 ==
 * 0; w 16-byte aligned, device): a group's scale is its largest magnitude / 7
 * rounded to bf16, its codes value / scale rounded half to even, at most 7 in
 * magnitude.  A group of zeros, or whose scale rounds to 0, has codes 0; one
 * with an infinity or NaN has scale NaN.  The last group of a row may be short.
 * w must not overlap the tiles. */
bloom_status bloom_op_w4_quantize(const void *w, int64_t ld, const bloom_w4 *out, void *stream);

/* Read the weights back: code * scale rounded to bf16, [n][k] at w (rows ld
 * apart, as above).  For prompts: widen a matrix once, then bloom_op_gemm. */
bloom_status bloom_op_w4_read(const bloom_w4 *in, void *w, int64_t ld, void *stream);

/* The linear layer of a decode step over 4-bit weights: y[m][i] = epilogue(sum_k
 * W[i][k] x[m][k] + bias[i]), W = code * scale, sums in float32.  x: bf16 [M][k],
 * rows ldx apart (ldx >= k, ldx % 8 == 0; 16-byte aligned); bias: bf16 [n] or
 * NULL; y: bf16 (y_f32 = 0) or float (1) [M][n], rows ldy >= n apart, aligned to
 * its elements; epilogue as bloom_op_linear (BLOOM_EPI_RESID adds to y in
 * place).  M up to 2^20; the weights are read once for every 64 tokens.  An
 * activation smaller than 2^-31 of the largest of its token (up to 8 tokens: of
 * its token's 256 columns 256 i .. 256 i + 255) is taken to within 2^-39 of that
 * one; others exactly.  That largest one goes into the sums as about 2^15: scales
 * from 2^-90 to 2^70 neither lose bits there nor overflow.
 * A token with an infinity or NaN among its activations has NaN outputs.  y
 * must not overlap x, the tiles or the bias.
 * `flag`: as for the 8-bit cache; bit 8: a bounded wait expired, the outputs
 * that depend on it are NaN. */
bloom_status bloom_op_linear_w4(const bloom_w4 *w, const void *x, int64_t ldx, int32_t M,
                                const void *bias, int32_t epilogue, void *y, int64_t ldy,
                                int32_t y_f32, void *workspace, size_t workspace_bytes,
                                int32_t *flag, void *stream);

/* Bytes of workspace that a call with M tokens needs (16-byte aligned device memory, its
 * content meaningless before and after; calls whose work overlaps need one each): 0 up to
 * 8 tokens, and on bad arguments. */
size_t bloom_op_linear_w4_workspace(const bloom_w4 *w, int32_t M);

/* Bound of the waits of this thread's calls of bloom_op_linear_w4 from now on, in
 * nanoseconds; 0 (the default): about two seconds. */
bloom_status bloom_op_linear_w4_wait_ns(int32_t wait_ns);

/* Tied LM head with fused argmax: logits[m][v] = x[m] . E[v]; out_tokens[m] =
 * lowest index of the row maximum of the float32 logits; out_logits may be
 * NULL.  x bf16 [M][K], E bf16 [V][K]. */
bloom_status bloom_op_lmhead_argmax(const void *x, const void *emb, int32_t M, int32_t V,
                                    int32_t K, int32_t *out_tokens, float *out_logits,
                                    void *stream);

/* ------------------------------------------------------------------------
 * Allocation-free variant (no counterpart on the pages: an addition of this
 * library).
 * ------------------------------------------------------------------------ */

/* Same result as bloom_op_lmhead_argmax, but the call allocates nothing: the
 * kernel's scratch (a completion ticket and one running maximum per row) is a
 * fixed array inside the library, present on every GPU that loads it until the
 * process exits.  For callers that cannot allocate device memory on the call
 * path (cudaMalloc / cudaFree may synchronise the device or fail under memory
 * pressure; a framework's caching allocator may own all GPU memory; serving
 * loops may forbid allocation between requests).
 *  - M <= 256 rows; larger M returns BLOOM_E_CAPACITY and launches nothing.
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current and keeps it for the
 *    process; make that first call before any stream capture, and make no call
 *    after a cudaDeviceReset of that device (the kept address would be stale).
 *  - Each call clears the part of the array it uses (cudaMemsetAsync on
 *    `stream`) before its kernel; calls whose work overlaps on the GPU (other
 *    streams, other threads) share the array and race, so serialise them. */
bloom_status bloom_op_lmhead_argmax_noalloc(const void *x, const void *emb, int32_t M,
                                            int32_t V, int32_t K, int32_t *out_tokens,
                                            float *out_logits, void *stream);

#ifdef __cplusplus
}
#endif
#endif
