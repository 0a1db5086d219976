/*
 * graphdec.h -- C ABI of the captured, constant-shape decode step on one GPU.
 *
 * What the library does.  A Llama-style pre-norm decoder step (embedding;
 * per layer RMSNorm, QKV projection, RoPE, K/V write at the slot position,
 * attention that sweeps the fixed KV capacity `cap` under an iota-vs-pos mask,
 * output projection, RMSNorm, SwiGLU MLP; final RMSNorm, LM head, greedy
 * argmax) is recorded once into a CUDA graph and replayed per token.  Between
 * replays the host only rewrites the slot buffers (Token, Pos, and for paged
 * KV the SlotMap page table and the WriteMap target slot).  Sources on the
 * pages: "Execution" (sections "Why capture", "A constant-shape decode graph",
 * "Slot buffers", "Per backend" -- PTX row, "Failure handling"),
 * "Backends" (section "PTX (NVIDIA)"), "Models, Registry and the Driver"
 * (sections "The Model" -- StepShape, "Shared components" -- standard_stack).
 *
 * Conventions shared by every call.
 *   - Every call returns an int status (dec_status); DEC_OK == 0.  After a
 *     failure, dec_last_error() returns a NUL-terminated message owned by the
 *     handle (valid until the next call on that handle); dec_last_error(NULL)
 *     gives the message of the last failed call without a handle (dec_init,
 *     dec_kv8_*, dec_w4_*) on the calling thread.
 *   - Pointers marked "device" are CUDA device addresses on the handle's GPU;
 *     "host" pointers are ordinary (pageable or pinned) host memory.  The
 *     library never frees memory it did not allocate.
 *   - A handle is thread-compatible, not thread-safe: one thread at a time.
 *     All device work of a handle runs on one CUDA stream.
 *   - Row-major everywhere.  Matrices use the nn.Linear layout [out, in].
 *   - Failure states ("Execution", section "Failure handling"): a device-side
 *     check that fails (token, position or map value out of range) sets a bit
 *     in the step's error word; the step's results are discarded, the call
 *     returns DEC_E_DEVICE_FAULT and the handle needs dec_reset_state() before
 *     it steps again (DEC_E_NEEDS_RESET until then).  A CUDA error or a wait
 *     that outlasts the configured timeout poisons the handle: every later
 *     call except dec_last_error / dec_stats / dec_destroy returns
 *     DEC_E_POISONED without touching the device.
 */
#ifndef GRAPHDEC_H
#define GRAPHDEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DEC_ABI_VERSION 1

typedef struct dec_handle dec_handle;

typedef enum dec_status {
    DEC_OK = 0,
    DEC_E_INVALID = 1,       /* malformed argument or configuration */
    DEC_E_UNSUPPORTED = 2,   /* well-formed, but this library cannot run it (message names the field) */
    DEC_E_RANGE = 3,         /* a token, position or map entry outside its range (host check) */
    DEC_E_STATE = 4,         /* call out of order (e.g. dec_step before dec_capture) */
    DEC_E_CUDA = 5,          /* CUDA runtime error; the handle is poisoned */
    DEC_E_OOM = 6,           /* device allocation failed or workspace too small */
    DEC_E_DEVICE_FAULT = 7,  /* a device-side check failed; see dec_stats.last_fault */
    DEC_E_NEEDS_RESET = 8,   /* an earlier step failed; call dec_reset_state */
    DEC_E_POISONED = 9,      /* the handle saw a CUDA error or a timeout; only dec_destroy helps */
    DEC_E_TIMEOUT = 10       /* a device wait outlasted wait_timeout_ms; the handle is poisoned */
} dec_status;

/* bits of the device error word (dec_stats.last_fault) */
#define DEC_FAULT_TOKEN     0x1u  /* Token[r] outside [0, vocab) */
#define DEC_FAULT_POS       0x2u  /* Pos[r] outside [0, cap) */
#define DEC_FAULT_WRITE_MAP 0x4u  /* WriteMap[r] outside [0, num_pages * page_size) */
#define DEC_FAULT_SLOT_MAP  0x8u  /* a SlotMap entry outside [0, num_pages) */
#define DEC_FAULT_WAIT      0x10u /* an in-kernel wait on another CTA or on a copy gave up (bounded poll) */
#define DEC_FAULT_SCALE     0x20u /* a scale byte of an 8-bit K/V block outside [27, 227] */

/* E4M3 is a K/V store's type only: one byte a value with a power-of-two scale for
 * each block of positions and head, see "The 8-bit K/V cache" below. */
typedef enum dec_dtype { DEC_DTYPE_F32 = 0, DEC_DTYPE_BF16 = 1, DEC_DTYPE_E4M3 = 2 } dec_dtype;

/* KV layouts ("Execution", section "A constant-shape decode graph"):
 *   CONTIGUOUS: per layer K and V of shape [rows, n_kv_heads, cap, head_dim];
 *               the step writes position Pos[r] (a DynamicUpdateSlice).
 *   PAGED:      per layer a pool [num_pages, n_kv_heads, page_size, head_dim]
 *               for K and one for V; logical position j of row r lives in
 *               slot SlotMap[r][j / page_size] * page_size + j % page_size, and
 *               the step scatters the new K/V to slot WriteMap[r]
 *               (a ScatterUpdate through Slot::WriteMap). */
typedef enum dec_kv_layout { DEC_KV_CONTIGUOUS = 0, DEC_KV_PAGED = 1 } dec_kv_layout;

/* How the captured step executes (chosen before dec_capture):
 *   GRAPH       the pages' strategy: the step's dispatch sequence (embedding,
 *               5 fused kernels per layer, head) recorded into one CUDA graph
 *               with programmatic dependent launches ("Execution", "Per
 *               backend", PTX row);
 *   PERSISTENT  the step as one cooperative kernel captured as the graph's
 *               single node; phases separated by grid-wide dependency counters
 *               and one continuous weight/KV stream per SM (the pages' possible
 *               future megakernel strategy).  Same arithmetic, other fp32
 *               summation order: results agree with GRAPH within the parity
 *               tolerances, not bit for bit; replay and eager runs of one
 *               strategy are bit-identical.  Available for bf16 weights and
 *               KV with the 8B-shape or 1B-class layer shapes at rows = 1
 *               (contiguous or paged K/V), and with the 1B-class shape at
 *               rows = 2 or 4 with contiguous K/V (DEC_E_UNSUPPORTED at
 *               capture otherwise). */
typedef enum dec_strategy { DEC_STRATEGY_GRAPH = 0, DEC_STRATEGY_PERSISTENT = 1 } dec_strategy;

/* Which K/V positions the attention of the captured step reads:
 *   CAP  the method's constant-shape sweep of [0, cap) with the position mask
 *        ("Execution", "A constant-shape decode graph": attention always
 *        sweeps [cap]; a mask computed from Slot::Pos against an iota hides
 *        the positions after pos) -- the default;
 *        (an e4m3 store's attention reads what the token sees, under either)
 *   POS  the same captured graph and grid, but each split stops loading K/V
 *        tiles after the one holding pos (a split that starts after pos loads
 *        none).  The tiles it skips are fully masked, and the kernel already
 *        does no arithmetic on a 16-key block without a visible key, so the
 *        results are bit-identical to CAP; only the bytes read shrink from the
 *        capacity to the positions up to pos. */
typedef enum dec_kv_sweep { DEC_SWEEP_CAP = 0, DEC_SWEEP_POS = 1 } dec_kv_sweep;

/* Model configuration.  RMSNorm is x / sqrt(mean(x^2) + rms_eps) * g; RoPE is
 * the half-split rotation of pairs (i, i + head_dim/2) by pos * rope_theta^(-2i/head_dim);
 * attention scale is 1/sqrt(head_dim); q head i reads kv head i / (n_heads / n_kv_heads). */
typedef struct dec_config {
    int32_t n_layers;
    int32_t d_model;
    int32_t n_heads;        /* query heads */
    int32_t n_kv_heads;     /* key/value heads; must divide n_heads */
    int32_t head_dim;       /* even */
    int32_t ffn_hidden;     /* SwiGLU hidden width */
    int32_t vocab;
    int32_t weight_dtype;   /* dec_dtype of every weight (matrices, embeddings, norm gains) */
    int32_t kv_dtype;       /* dec_dtype of the stored K/V; E4M3: head_dim 64 or 128, DEC_STRATEGY_GRAPH,
                             * a cap (contiguous) or pages that are multiples of 16, new K/V stored by
                             * dec_kv8_append's rules; only positions that a token sees are read */
    int32_t device;         /* CUDA device ordinal */
    double rms_eps;
    double rope_theta;
    int64_t wait_timeout_ms;  /* bound on every device wait; <= 0 means 600000 (600 s) */
} dec_config;

/* Weight roles ("Execution": load_weights binds each weight by its typed role;
 * a weight no binding names stays unbound and dec_capture refuses to run). */
typedef enum dec_role {
    DEC_W_EMBED = 0,       /* [vocab, d_model]                     global (layer = -1) */
    DEC_W_ATTN_NORM = 1,   /* [d_model]                            per layer */
    DEC_W_Q = 2,           /* [n_heads * head_dim, d_model]        per layer */
    DEC_W_K = 3,           /* [n_kv_heads * head_dim, d_model]     per layer */
    DEC_W_V = 4,           /* [n_kv_heads * head_dim, d_model]     per layer */
    DEC_W_O = 5,           /* [d_model, n_heads * head_dim]        per layer */
    DEC_W_FFN_NORM = 6,    /* [d_model]                            per layer */
    DEC_W_GATE = 7,        /* [ffn_hidden, d_model]                per layer */
    DEC_W_UP = 8,          /* [ffn_hidden, d_model]                per layer */
    DEC_W_DOWN = 9,        /* [d_model, ffn_hidden]                per layer */
    DEC_W_FINAL_NORM = 10, /* [d_model]                            global */
    DEC_W_LM_HEAD = 11,    /* [vocab, d_model]                     global */
    DEC_W_NROLES = 12
} dec_role;

typedef struct dec_weight {
    int32_t role;      /* dec_role */
    int32_t layer;     /* 0 .. n_layers-1 for per-layer roles, -1 for global roles */
    int32_t dtype;     /* must equal dec_config.weight_dtype */
    int32_t reserved;  /* 0 */
    int64_t rows;      /* shape [rows, cols]; a gain vector of length n is [n, 1] */
    int64_t cols;
    const void *data;  /* device, 16-byte aligned, borrowed: must outlive the handle */
} dec_weight;

typedef struct dec_stats {
    int64_t steps;            /* completed dec_step / dec_wait calls */
    int64_t replays;          /* graph launches */
    int64_t eager_steps;      /* kernel sequences launched without the graph */
    int32_t kernels_per_step; /* kernel launches recorded per step */
    int32_t graph_nodes;      /* nodes of the instantiated graph */
    int32_t attn_splits;      /* KV splits per (row, kv head) */
    int32_t attn_split_len;   /* positions per split */
    uint32_t last_fault;      /* error word of the last failed step (DEC_FAULT_* bits) */
    int32_t state;            /* 0 ready, 1 needs reset, 2 poisoned */
    int32_t captured;         /* 1 after dec_capture */
    int32_t rows;
    int32_t cap;
    int32_t kv_layout;
    int32_t strategy;         /* dec_strategy of the capture */
    int32_t reserved;
    double last_step_us;      /* host wall time of the last dec_step */
    int64_t workspace_bytes;  /* device bytes the capture uses (KV included) */
    int64_t kv_bytes;         /* device bytes of K and V over all layers, an e4m3 store's scales included */
} dec_stats;

/* Create a handle for `cfg` on cfg->device ("Execution", executor contract:
 * one engine per target, set up before any weight is bound; the handle plays
 * the executor object and every later call goes through it).  Validates the
 * configuration (DEC_E_INVALID / DEC_E_UNSUPPORTED naming the field, like the
 * planner's refusals) before touching the GPU; DEC_E_CUDA if the device cannot
 * be selected.  *out receives the handle, or NULL on failure; the caller owns
 * it and releases it with dec_destroy. */
int dec_init(const dec_config *cfg, dec_handle **out);

/* Bind `n` weights by role ("Execution": load_weights(store, map)).  May be
 * called several times before dec_capture; a later binding of the same
 * (role, layer) replaces the earlier one.  Shapes and dtypes are checked
 * against the configuration (DEC_E_INVALID).  The library reads the weights in
 * place: nothing is copied. */
int dec_load_weights(dec_handle *h, const dec_weight *w, size_t n);

struct dec_w4_binding;

/* Bind `n` matrices in 4 bits by role (the format is at dec_w4_weight below):
 * Q, K, V, O, GATE, UP and DOWN of a layer, all seven or none, and LM_HEAD (layer
 * -1).  A later binding of a role replaces an earlier one of either kind.  Norm
 * gains and embeddings stay in weight_dtype.  Q, K and V of a layer have one group,
 * and so have GATE and UP.  Read in place like the others; the step's products are
 * dec_w4_linear's and dec_w4_glu's.  DEC_STRATEGY_GRAPH only, and with layers in 4
 * bits no dec_prefill_block (DEC_E_UNSUPPORTED there; dec_prefill takes them). */
int dec_load_w4(dec_handle *h, const struct dec_w4_binding *w, size_t n);

/* Device bytes that dec_capture needs for this shape (KV store, slots,
 * activations, attention partials, RoPE table): the preallocated Storage::State
 * buffers of capacity cap per layer plus the step's intermediates ("Execution",
 * section "A constant-shape decode graph": K and V are preallocated to cap).
 * Host-only (no device call).  *bytes (host) receives the size; DEC_E_INVALID
 * for a configuration dec_init would refuse or a shape dec_capture would refuse. */
int dec_workspace_size(const dec_config *cfg, int32_t cap, int32_t rows, int32_t kv_layout,
                       int32_t page_size, int32_t num_pages, size_t *bytes);

/* Allocate the step's buffers, run the kernel sequence once eagerly (checks),
 * clear the state, and record the sequence into one CUDA graph that serves
 * every position 0 <= pos < cap ("Execution", section "A constant-shape decode
 * graph": grids and buffer addresses stay constant, so one capture serves
 * every position up to cap).  One capture per handle ("Models, Registry and
 * the Driver": one entry per step shape; capacity is part of the shape).
 *   cap        KV capacity (positions per row), >= 1
 *   rows       sequences stepped together, 1 .. 8
 *   kv_layout  dec_kv_layout
 *   page_size, num_pages  paged layout only (cap % page_size == 0,
 *              rows * cap / page_size <= num_pages); ignored for contiguous
 *   workspace  device buffer of >= dec_workspace_size bytes, 256-byte aligned,
 *              owned by the caller and kept until dec_destroy; NULL: the library
 *              allocates (and frees at dec_destroy)
 *   stream     cudaStream_t to run on; NULL: the library creates its own.
 *              The legacy default stream cannot be captured and is refused.
 * All bound weights must be present (DEC_E_INVALID names the first missing). */
int dec_capture(dec_handle *h, int32_t cap, int32_t rows, int32_t kv_layout, int32_t page_size,
                int32_t num_pages, void *workspace, size_t workspace_bytes, void *stream);

/* Rewrite the paged read map ("Execution", section "Slot buffers":
 * Slot::SlotMap).  map: host, [rows, cap / page_size] int32 page ids, each in
 * [0, num_pages) (DEC_E_RANGE otherwise).  Takes effect from the next step.
 * DEC_E_STATE for a contiguous capture. */
int dec_set_slot_map(dec_handle *h, const int32_t *map);

/* One decode step of every row ("Execution", section "Per backend", PTX row:
 * write slots, launch the graph, copy results back, wait).
 *   tokens     host [rows], each in [0, vocab)
 *   pos        host [rows], each in [0, cap): the absolute position of the token
 *   write_map  host [rows] target slot for paged KV, or NULL to derive it from
 *              the slot map as SlotMap[r][pos/page]*page + pos%page; ignored
 *              for contiguous KV
 *   logits_out host [rows, vocab] fp32, or NULL
 *   ids_out    host [rows] greedy token ids (largest logit, lowest index on
 *              ties), or NULL
 *   nonfinite_out host [rows], 1 if any logit of the row is NaN or Inf, or NULL
 * Host-side range checks return DEC_E_RANGE before anything is launched. */
int dec_step(dec_handle *h, const int32_t *tokens, const int32_t *pos, const int32_t *write_map,
             float *logits_out, int32_t *ids_out, uint8_t *nonfinite_out);

/* Asynchronous half of a step: copy the slot record (device, [3 * rows]
 * int32: tokens, then positions, then write map) into the slot buffers and
 * launch the step, without waiting and without host-side range checks (the
 * device checks still run).  Results stay on the device until dec_wait. */
int dec_launch(dec_handle *h, const int32_t *dev_slots);

/* Wait (bounded by wait_timeout_ms) for the launched steps and copy the last
 * step's results back; any pointer may be NULL.  Returns DEC_E_DEVICE_FAULT if
 * the last step's error word is non-zero. */
int dec_wait(dec_handle *h, float *logits_out, int32_t *ids_out, uint8_t *nonfinite_out);

/* Chained greedy steps ("Models, Registry and the Driver", section "The
 * Driver": RowWork::Chain -- with no guided row, several decode steps run back
 * to back, the device feeds each step's pick to the next and the host waits
 * once).  Step 0 runs tokens at pos; step i > 0 runs, for every row, the
 * greedy id of step i - 1 at pos + i.  Each step is one replay of the recorded
 * step followed by a one-CTA kernel that records the ids and writes the next
 * step's Token, Pos and (paged) WriteMap slots from the device; the host
 * copies the histories back once and waits once.
 *   n_steps       1 .. DEC_CHAIN_MAX_STEPS
 *   tokens, pos   host [rows], as for dec_step; pos[r] + n_steps <= cap
 *                 (DEC_E_RANGE otherwise, before anything is launched)
 *   ids_out       host [n_steps, rows]: the greedy id of each step (required)
 *   nonfinite_out host [n_steps, rows] non-finite flags, or NULL
 * Paged KV takes every WriteMap from the current slot map.  A device check
 * that fails in any step of the chain returns DEC_E_DEVICE_FAULT (results
 * discarded, reset needed).  The logits of the last step stay on the device
 * (dec_logits_ptr). */
#define DEC_CHAIN_MAX_STEPS 4096
int dec_chain(dec_handle *h, int32_t n_steps, const int32_t *tokens, const int32_t *pos, int32_t *ids_out,
              uint8_t *nonfinite_out);

/* Multi-token prefill of ONE sequence ("Models, Registry and the Driver",
 * section "The Model": a step shape is rows x new tokens; positions are
 * absolute, so a prefill is a step continuing from a position).  The n tokens
 * at positions pos0 .. pos0 + n - 1 run through the recorded paged step in
 * chunks of `rows` tokens: in each chunk row t is position pos0 + c + t of the
 * sequence, every row reads and writes the sequence's pages, and every row's
 * K/V is stored before any row's attention reads the pages.  Afterwards the
 * sequence's K/V for those positions is in its pages, and the caller's slot
 * map is in place again.
 *   pages       host [cap / page_size] page ids of the sequence, each in
 *               [0, num_pages)
 *   tokens      host [n], each in [0, vocab)
 *   pos0        first position; pos0 + n <= cap (DEC_E_RANGE otherwise)
 *   logits_out  host [vocab] fp32 logits after the last token, or NULL
 *   id_out      host, the greedy id after the last token, or NULL
 * Needs a paged graph capture of 2..8 rows with bf16 or e4m3 K/V
 * (DEC_E_UNSUPPORTED otherwise).  Per token the arithmetic equals a decode step
 * of that token, so the chunking does not change any result -- except that with
 * e4m3 K/V a chunk's later tokens may have raised the scale of a block, and so
 * rounded its earlier tokens again, before the earlier ones attend to them. */
int dec_prefill(dec_handle *h, const int32_t *pages, const int32_t *tokens, int32_t n, int32_t pos0,
                float *logits_out, int32_t *id_out);

/* Multi-token prefill of ONE sequence as a block step ("Models, Registry and
 * the Driver", section "The Model": a step shape is rows x new tokens;
 * positions are absolute, so a prefill is a step continuing from a position).
 * The n tokens at positions pos0 .. pos0 + n - 1 run layer by layer in passes
 * of up to 1024 tokens (blocks of 128 for the tensor cores): per layer the
 * projections are dense contractions on the tensor cores
 * (tcgen05.mma, bf16 weights, activations as bf16 hi + lo parts, fp32
 * accumulation), attention is causal over every position up to each token
 * (online softmax, fp32), and every layer's K/V of the n positions is written
 * into the sequence's store (rounded to bf16, or by dec_kv8_append's rules).  The last token's hidden state
 * then goes through the captured step's final RMSNorm, LM head and argmax.
 *   row         contiguous K/V: the capture row whose store holds the
 *               sequence (0 .. rows-1); ignored for paged K/V
 *   pages       paged K/V: host [cap / page_size] page ids of the sequence, each
 *               in [0, num_pages); NULL for contiguous K/V
 *   tokens      host [n], each in [0, vocab)
 *   pos0        first position; pos0 + n <= cap (DEC_E_RANGE otherwise)
 *   logits_out  host [vocab] fp32 logits after the last token, or NULL
 *   id_out      host, the greedy id after the last token, or NULL
 * Positions before pos0 must already hold the sequence's K/V (from steps or an
 * earlier prefill).  Any capture with bf16 weights and bf16 or e4m3 K/V whose
 * shape has head_dim 64 or 128, d_model, n_heads * head_dim and ffn_hidden
 * multiples of 64, d_model <= 8192 and with bf16 K/V n_heads / n_kv_heads of 2
 * or 4 and (paged) pages of at least 8 tokens (DEC_E_UNSUPPORTED otherwise).  The
 * first call allocates the block's device buffers (cudaMalloc, kept until
 * dec_destroy); the call is synchronous (bounded wait) and must not be
 * captured.  Results agree with stepping the tokens one at a time within the
 * parity tolerances, not bit for bit (other arithmetic, other summation
 * order).  The captured step's slot buffers are untouched; its logits buffer
 * holds this call's logits afterwards. */
int dec_prefill_block(dec_handle *h, int32_t row, const int32_t *pages, const int32_t *tokens, int32_t n,
                      int32_t pos0, float *logits_out, int32_t *id_out);

/* Sampling suffix beyond greedy ("Models, Registry and the Driver", section
 * "The Driver": Head::Sample -- greedy or temperature / top-k / top-p /
 * min-p, optional top-n logprobs).  For each row of a step:
 *   candidates  the top_k tokens of largest logit (ties: lower index);
 *   weights     q = exp((logit - max logit) / temperature);
 *   kept        the shortest prefix of the candidates, by logit, whose weight
 *               reaches top_p of the candidates' total, and only candidates
 *               with q >= min_p (relative to the largest probability);
 *   pick        inverse CDF over the kept prefix at u = the top 53 bits of
 *               splitmix64 at counter (row << 32 | Pos[row]) of `seed`,
 *               i.e. mix64(seed + (counter + 1) * 0x9E3779B97F4A7C15);
 *   logprobs    logit - max - log(sum over the vocabulary of exp(logit - max))
 *               of the n_logprobs tokens of largest logit.
 * temperature = 0 picks the greedy id. */
#define DEC_SAMPLER_MAX_TOP_K 1024
#define DEC_LOGPROBS_MAX 8
typedef struct dec_sampler {
    float temperature;   /* >= 0; 0: greedy */
    int32_t top_k;       /* 1 .. DEC_SAMPLER_MAX_TOP_K when temperature > 0 */
    float top_p;         /* (0, 1]; 1: no top-p cut */
    float min_p;         /* [0, 1); 0: no min-p cut */
    uint64_t seed;
    int32_t n_logprobs;  /* 0 .. DEC_LOGPROBS_MAX */
    int32_t reserved;
} dec_sampler;

/* Before dec_capture: a non-NULL sampler records the sampling kernel after the
 * head in the step (NULL: greedy only, nothing recorded).  After dec_capture:
 * rewrites the sampler's parameters in place for the coming steps (a slot
 * buffer, no re-capture); DEC_E_STATE if no sampler was recorded.  With a
 * sampler recorded, the ids returned by dec_step / dec_wait and fed forward by
 * dec_chain are the sampled ids.  DEC_E_INVALID for parameters out of range. */
int dec_set_sampler(dec_handle *h, const dec_sampler *s);

/* Top-n logprobs of the last completed step: ids_out and logprobs_out host
 * [rows, n], n <= the sampler's n_logprobs (DEC_E_INVALID otherwise). */
int dec_logprobs(dec_handle *h, int32_t n, int32_t *ids_out, float *logprobs_out);

/* Choose the execution strategy (dec_strategy) for the coming dec_capture;
 * DEC_E_STATE after capture.  Default DEC_STRATEGY_GRAPH. */
int dec_set_strategy(dec_handle *h, int32_t strategy);

/* Choose the K/V sweep (dec_kv_sweep) of the coming dec_capture; DEC_E_STATE
 * after capture, DEC_E_INVALID for an unknown value.  Default DEC_SWEEP_CAP.
 * DEC_SWEEP_POS needs the GRAPH strategy and a tensor-core attention kernel
 * (bf16 or e4m3 K/V, head_dim 64 or 128): dec_capture returns DEC_E_UNSUPPORTED
 * otherwise.  It also applies to dec_attention on the same handle. */
int dec_set_kv_sweep(dec_handle *h, int32_t sweep);

/* Attention within a window for the coming dec_capture (DEC_E_STATE after it):
 * a token at position i sees j <= i with j > i - window or j < sinks; window 0
 * (the default): every j <= i.  DEC_E_INVALID for negative values.  Needs an
 * e4m3 K/V store (dec_capture returns DEC_E_UNSUPPORTED otherwise).  Also
 * applies to dec_attention, dec_prefill and dec_prefill_block on the handle. */
int dec_set_window(dec_handle *h, int32_t window, int32_t sinks);

/* 1: later steps launch the recorded kernel sequence directly on the stream
 * instead of replaying the graph (same kernels, same arguments); 0: replay. */
int dec_set_eager(dec_handle *h, int32_t eager);

/* Zero the KV store, the slot buffers and the error word, and clear the
 * needs-reset state ("Execution", section "Failure handling": step refuses
 * until reset_state clears it).  A poisoned handle stays poisoned. */
int dec_reset_state(dec_handle *h);

/* Device address and byte size of one layer's K (which = 0) or V (which = 1)
 * store, in the layout of the capture's dec_kv_layout: the carried state that
 * the pages' reference evaluation returns beside the primary output and that
 * parity covers element by element ("Execution", section "Verification", tier
 * 2: every output and carried state).  For tests that pre-fill or inspect it.
 * *ptr (host) receives a device pointer owned by the handle (valid until
 * dec_destroy); *bytes (host, optional) its size.  DEC_E_STATE before
 * dec_capture, DEC_E_INVALID for a bad layer or which. */
int dec_kv_ptr(dec_handle *h, int32_t layer, int32_t which, void **ptr, size_t *bytes);

/* E4M3 store: device address and byte size (optional) of the scales of one
 * layer's K (which = 0) or V (which = 1), one byte for each block of *block
 * positions (optional) and head: [rows or num_pages, n_kv_heads, positions /
 * block], exponent + 127.  block is 64, 32 or 16, the largest that divides the
 * cap (contiguous) or the page.  Like dec_kv_ptr otherwise; DEC_E_STATE for
 * another K/V type. */
int dec_kv_scale_ptr(dec_handle *h, int32_t layer, int32_t which, void **ptr, size_t *bytes, int32_t *block);

/* One layer's decode attention as a standalone operation, on the caller's
 * buffers ("Execution", section "A constant-shape decode graph"): rotates q and
 * k by RoPE at pos[r], writes the rotated k and v (rounded to the KV dtype)
 * into this layer's KV store at pos[r] (paged: at the slot of the current
 * write map), and attends over the full capacity with positions after pos[r]
 * masked.  Runs on the handle's stream and waits (bounded).
 *   layer  0 .. n_layers-1
 *   qkv    device fp32 [rows, (n_heads + 2 * n_kv_heads) * head_dim]: q, then k,
 *          then v of every row, before RoPE
 *   pos    device int32 [rows], each in [0, cap)
 *   out    device fp32 [rows, n_heads * head_dim]
 * The split partials use the handle's workspace.  DEC_E_DEVICE_FAULT if a
 * device check fails (the handle then needs dec_reset_state). */
int dec_attention(dec_handle *h, int32_t layer, const float *qkv, const int32_t *pos, float *out);

/* dec_attention without any allocation.  Same operation, arguments and
 * results as dec_attention; the split scratch (partials and completion
 * counters) lives in a fixed device array inside the library instead of the
 * handle's workspace, so this call allocates nothing.  It is for callers that
 * cannot allocate device memory where they run attention: a serving process
 * that reserved its whole device-memory budget up front (weights and KV cache
 * sized to fill the GPU) and has nothing left to hand out per call, and code
 * whose latency cannot absorb cudaMalloc / cudaFree, which may synchronise the
 * whole device.  Like dec_attention it runs on the handle's stream and waits
 * (bounded) for its result before returning.  The pages have no counterpart of
 * this entry point.
 * Limits: the array holds 2^19 fp32 partials and 1024 counters (about 2 MiB); a
 * shape that needs more (rows * n_heads * splits * (head_dim + 4) floats)
 * returns DEC_E_UNSUPPORTED and leaves the handle usable, as does an e4m3
 * store (its attention has scratch in the capture's workspace).  Every GPU that loads
 * the library keeps the array until the process exits.  All calls on a device
 * share the array (it keeps the last call's contents; the counters are cleared
 * on entry), so calls that overlap on the GPU race: serialise them.  The first
 * call on a device looks up the array's device address (once per device, kept
 * for the life of the process; a cudaDeviceReset invalidates it together with
 * every handle); make that first call before any stream capture. */
int dec_attention_static(dec_handle *h, int32_t layer, const float *qkv, const int32_t *pos, float *out);

/* ---- The 8-bit K/V cache ----
 * K and V of a batch of sequences in e4m3 (one byte a value: half of bf16's
 * bytes to hold and to read), with one power-of-two scale for each block of
 * scale_block consecutive positions of one K/V head.  A stored byte x8 in a
 * block with scale byte s stands for x8 * 2^(s - 127); scale bytes that
 * dec_kv8_append writes lie in [87, 187]; a caller who fills a cache by other
 * means keeps them in [27, 227] (2^-100 .. 2^100: the attention's sums are fp32).
 *
 * These calls stand beside dec_attention for callers who keep their own cache.
 * They take no handle, only launch kernels on the caller's stream (NULL: the
 * legacy default stream), neither wait nor allocate, and may be recorded into
 * a graph; lengths, page table and token ranges are read from device memory
 * when the kernels run, so one recorded graph serves every step.  The current
 * device is put back before they return.  Messages: dec_last_error(NULL).
 *
 * Layout: the pools are [num_pages, n_kv_heads, page_size, head_dim] like the
 * paged K/V of a capture; position j of row r lies in page
 * pages[r * pages_per_row + j / page_size] at j % page_size (pages = NULL: in
 * page r * pages_per_row + j / page_size, the contiguous layout).  Rows may
 * share pages that no append writes to.  K is stored as the caller gives it
 * (rotated by RoPE already).
 *   head_dim     64 or 128           scale_block  16, 32, 64 or 128
 *   page_size    a multiple of scale_block
 *   rows         1 .. 1024; pages_per_row * page_size <= 2^30 */
typedef struct dec_kv8_cache {
    void *k, *v;                 /* device, 16-byte aligned: e4m3 pools */
    uint8_t *k_scale, *v_scale;  /* device: [num_pages, n_kv_heads, page_size / scale_block] */
    const int32_t *pages;        /* device [rows, pages_per_row], or NULL */
    int32_t rows, pages_per_row, page_size, num_pages, n_kv_heads, head_dim, scale_block;
    int32_t device;              /* CUDA device ordinal of all of it */
} dec_kv8_cache;

/* Which tokens a call works on.  Tokens of all rows are packed: row r has the
 * n = q_start[r + 1] - q_start[r] tokens from q_start[r] on, at the positions
 * kv_len[r] - n .. kv_len[r] - 1.  Rows may have none.  A token whose position
 * is negative (kv_len[r] < n: an idle row of a padded batch has kv_len 0) is
 * not stored and sees nothing.  Packed tokens that belong to no row are left
 * as they are.
 * A row with q_start or kv_len out of range (not 0 <= q_start[r] <= q_start[r+1]
 * <= total, more than max_new tokens, kv_len outside [0, pages_per_row *
 * page_size]) sets DEC_FAULT_POS in *err and is skipped whole; a page id that
 * is needed and outside [0, num_pages) sets DEC_FAULT_SLOT_MAP, and the page
 * counts as holding nothing.  DEC_FAULT_SCALE: attention met a scale byte outside
 * [27, 227]; the results of the row's tokens are not to be used.  DEC_FAULT_WAIT:
 * a copy or product never ended, and the call's results are not to be used. */
typedef struct dec_kv8_batch {
    const int32_t *q_start;      /* device [rows + 1], or NULL: one token for each row */
    const int32_t *kv_len;       /* device [rows]: positions of each row, this call's tokens included */
    uint32_t *err;               /* device: DEC_FAULT_* bits are added, never cleared */
    int32_t total;               /* packed tokens */
    int32_t max_new;             /* the most tokens of one row (sizes the launch) */
} dec_kv8_batch;

/* New K and V: [total, n_kv_heads, head_dim], heads side by side, tokens any
 * stride apart (elements; a multiple of 16 bytes): views into a packed QKV
 * matrix need no copy. */
typedef struct dec_kv8_new {
    const void *k, *v;           /* device, 16-byte aligned */
    int64_t k_stride, v_stride;
    int32_t dtype;               /* dec_dtype of k and v */
    int32_t reserved;            /* 0 */
} dec_kv8_new;

/* Store the batch's new K and V.  Each block that new tokens enter takes the
 * least exponent e with max |x| <= 448 * 2^e over its new finite values (at
 * least -40; at least the block's own if it holds earlier positions of the
 * row), and x is stored as e4m3(x * 2^-e), round to nearest even.  If e grew,
 * the block's earlier positions are rounded again at the new exponent.  NaN,
 * infinities and values over 448 * 2^60 are stored as NaN.  Positions behind
 * the row's end are left as they are; storing a position again (a rejected
 * draft) replaces it.  Two rows must not store into the same block in a call.
 * Results do not depend on scheduling. */
int dec_kv8_append(const dec_kv8_cache *cache, const dec_kv8_batch *batch, const dec_kv8_new *tokens, void *stream);

/* Attention of the batch's tokens over the cache (their own K and V stored
 * before): out = sum_j softmax_j(scale * q . k_j) v_j over the positions j that
 * the token at position i sees: j <= i and, with a window, j > i - window or
 * j < sinks.  A token that sees nothing gets zeros.  Query head a reads K/V
 * head a / (n_heads / n_kv_heads).  What a token does not see never reaches its
 * result, whatever bits it holds; a NaN that it sees does.  Scores, weights and
 * sums are held in fp32; with fp32 q the products are exact to about 2^-20, with
 * bf16 q the softmax weights to 2^-11 or finer, which is finer than the result.
 * That holds for each weight by itself, however small beside the largest (fp32's
 * range, about 2^-120).  Results do not depend on scheduling. */
typedef struct dec_kv8_attn {
    const void *q;               /* device [total, n_heads, head_dim], 16-byte aligned */
    void *out;                   /* device, the same shape and type; may not overlap q */
    int64_t q_stride, out_stride;   /* elements between tokens; a multiple of 16 bytes */
    int32_t dtype;               /* dec_dtype of q and out */
    int32_t n_heads;             /* n_heads / n_kv_heads <= 128 */
    int32_t window;              /* 0: none */
    int32_t sinks;               /* first positions that stay visible (with a window) */
    double scale;                /* 0: 1 / sqrt(head_dim) */
    void *workspace;             /* device, 16-byte aligned, dec_kv8_workspace bytes.  Zero-filled by the caller before
                                    its first use; every call leaves it ready for the next one on the same cache, of
                                    any size that it holds.  Calls that may overlap on the GPU need one each */
    size_t workspace_bytes;
} dec_kv8_attn;

int dec_kv8_attend(const dec_kv8_cache *cache, const dec_kv8_batch *batch, const dec_kv8_attn *attn, void *stream);

/* Bytes of workspace that dec_kv8_attend needs for these arguments (*bytes,
 * host).  Reads sizes only: the same for every content. */
int dec_kv8_workspace(const dec_kv8_cache *cache, const dec_kv8_batch *batch, const dec_kv8_attn *attn, size_t *bytes);

/* ---- 4-bit weights ----
 * A matrix [n, k] (nn.Linear layout) stored in 4 bits: codes -8 .. 7 in two's
 * complement, two in a byte (column 2i in the low half of byte i, 2i + 1 in the
 * high half; a row is k / 2 bytes, rows follow one another), and one bf16 scale
 * for each `group` consecutive columns of a row.  It stands for code * scale:
 * 4.125 bits a weight with groups of 128, a quarter of bf16's bytes to hold and,
 * in a decode step, to read.
 *
 * Like dec_kv8_* these calls take no handle, only launch kernels on the caller's
 * stream (NULL: the legacy default stream), neither wait nor allocate, and may be
 * recorded into a graph.  The current device is put back before they return.
 * Messages: dec_last_error(NULL).  A capture takes such matrices through
 * dec_load_w4.
 *   group   32, 64 or 128; k a multiple of it, at most 2^20
 *   n       >= 1, n * k <= 2^33 */
typedef struct dec_w4_weight {
    void *codes;                 /* device, 16-byte aligned: [n, k / 2] bytes */
    void *scales;                /* device, 2-byte aligned: bf16 [n, k / group] */
    int32_t n, k, group;
    int32_t device;              /* CUDA device ordinal of all of it */
} dec_w4_weight;

/* A matrix of a capture (dec_load_w4). */
typedef struct dec_w4_binding {
    int32_t role;                /* dec_role */
    int32_t layer;               /* 0 .. n_layers-1; -1 for LM_HEAD */
    dec_w4_weight w;             /* must outlive the handle */
} dec_w4_binding;

/* Store src [n, k] (f32 or bf16, rows src_stride elements apart, 16-byte aligned
 * like the stride) into w.  Over each group scale = bf16(max |x| / 7) and code =
 * x / scale to the nearest whole number, ties to even.  A group whose scale would
 * be below 2^-100 holds zeros at scale 0; a group with a NaN or an infinity has
 * scale NaN (and so gives NaN wherever it is used).  src, codes and scales do not
 * overlap. */
int dec_w4_quantize(const dec_w4_weight *w, const void *src, int64_t src_stride, int32_t dtype, void *stream);

/* The values that w stands for, [n, k] in f32 (exact) or bf16 (rounded once); rows
 * dst_stride elements apart, 16-byte aligned like the stride, and not over w's own
 * memory. */
int dec_w4_dequantize(const dec_w4_weight *w, void *dst, int64_t dst_stride, int32_t dtype, void *stream);

typedef enum dec_act { DEC_ACT_SILU = 0, DEC_ACT_GELU_TANH = 1 } dec_act;

/* One call's activations.  With a gain a = x / sqrt(mean(x^2) + eps) * gain, else
 * a = x.  out may be the residual itself (then with its stride); it overlaps
 * nothing else of the call. */
typedef struct dec_w4_call {
    const void *x;               /* device [tokens, k], 16-byte aligned */
    const void *gain;            /* device [k], 16-byte aligned, or NULL: no norm */
    const void *residual;        /* dec_w4_linear: device [tokens, n] of out's type, or NULL */
    void *out;                   /* device [tokens, n] */
    int64_t x_stride;            /* elements between tokens, a multiple of 16 bytes */
    int64_t residual_stride, out_stride;   /* at least n */
    int32_t tokens;              /* 0 .. 2^21; tokens * n and tokens * k <= 2^31 - 1 */
    int32_t x_dtype, gain_dtype, out_dtype;   /* F32 or BF16 each */
    int32_t act;                 /* dec_w4_glu: dec_act */
    int32_t reserved;            /* 0 */
    double eps;
    uint32_t *err;               /* device: DEC_FAULT_WAIT is added if a copy or product never ended (the call's results are
                                    not to be used); never cleared */
    void *workspace;             /* device, 256-byte aligned, dec_w4_workspace bytes (NULL where that is 0), of any content.
                                    Calls that may overlap on the GPU need one each */
    size_t workspace_bytes;
} dec_w4_call;

/* out[t, n] = residual[t, n] + sum_k W[n, k] a[t, k].
 *   Activations: bf16 ones enter exactly, fp32 ones and normed ones to about 2^-22
 * of each (and all to no less than 2^-39 of the token's largest; weights of more
 * than a few tokens to no less than 2^-38 of the row's largest scale).
 *   Sums: in fp32, off by less than 2^-18 of the result's size.  bf16 results of many
 * bf16 tokens without a gain come from sums of up to 32768 columns that the tensor
 * cores cut off: 2^-12 of the absolute values' sum at most, seen 4e-5 of the result's
 * size.
 *   For many bf16 tokens a gain or an fp32 result doubles the products: activations
 * that were normed to bf16 before the call are faster, and have 8 bits.
 *   Range: x * gain, x^2 and the sum of x^2 are fp32 values, so a normed token's
 * largest is below 2^63 / sqrt(k); without a gain, all finite values are taken.
 *   Results do not depend on scheduling nor on the values of other tokens, but their
 * last digits do on how many tokens a call has.  A token with a NaN or an infinity
 * gives NaN or infinities. */
int dec_w4_linear(const dec_w4_weight *w, const dec_w4_call *call, void *stream);

/* The first half of a gated feed-forward block: out[t, n] = act(gate_n . a_t) *
 * (up_n . a_t), gate and up of one shape and group.  silu(z) = z / (1 + e^-z);
 * gelu_tanh(z) = z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))). */
int dec_w4_glu(const dec_w4_weight *gate, const dec_w4_weight *up, const dec_w4_call *call, void *stream);

/* Bytes of workspace that dec_w4_linear (up = NULL) or dec_w4_glu needs for these
 * arguments (*bytes, host).  Reads sizes, types and whether there is a gain: of the
 * call's pointers and strides none is checked, and all but the gain may be NULL. */
int dec_w4_workspace(const dec_w4_weight *w, const dec_w4_weight *up, const dec_w4_call *call, size_t *bytes);

/* Device address of the logits [rows, vocab] fp32 of the last step. */
int dec_logits_ptr(dec_handle *h, float **ptr);

/* The CUDA stream the handle runs on (as a cudaStream_t). */
int dec_stream(dec_handle *h, void **stream);

/* Counters and state of the handle ("Execution", executor contract: stats).
 * Copies a dec_stats snapshot into *out (host); touches no device and works on
 * a poisoned handle.  DEC_E_INVALID for a NULL argument. */
int dec_stats_get(const dec_handle *h, dec_stats *out);

/* Device address of the paged read map [rows, cap / page_size] int32 (the
 * Slot::SlotMap buffer that the recorded kernels read, "Execution", section
 * "Slot buffers").  Introspection for tests: writing it directly bypasses
 * dec_set_slot_map's host range check, so the kernels' own check
 * (DEC_FAULT_SLOT_MAP) can be exercised.  Owned by the handle.  DEC_E_STATE
 * for a contiguous capture or before dec_capture. */
int dec_slot_map_ptr(dec_handle *h, int32_t **ptr);

/* Profiling hook: launch kernel `index` of the recorded step sequence alone,
 * eagerly, on the handle's stream (no slot write, no wait).  Order: 0 embedding;
 * per layer l: 1+5l RMSNorm+QKV, 2+5l attention (RoPE, K/V write, combine),
 * 3+5l output projection + residual, 4+5l RMSNorm+gate/up, 5+5l SwiGLU+down +
 * residual; last (5L+1) final RMSNorm + LM head + argmax.  The kernel reads and
 * writes the step's buffers as in a step (it changes the state).
 * pdl: 1 launches with the programmatic-serialization attribute as in the
 * graph, 0 with plain stream order.  *bytes (optional) receives the
 * algorithmic bytes one launch moves (weights read once + activations, or the
 * cap-swept K/V + q + partials for attention). */
int dec_launch_kernel(dec_handle *h, int32_t index, int32_t pdl, int64_t *bytes);

/* In-graph trace (profiling).  enable = 1 clears the stamps and makes every
 * recorded kernel stamp the device's global nanosecond timer at: its earliest
 * CTA entry, the latest CTA to pass the wait on the previous kernel, its
 * earliest CTA exit and its latest CTA exit; enable = 0 stops recording.
 * Stamps accumulate (min / max) over the steps run while enabled.  The
 * attention of an e4m3 K/V store does not stamp. */
int dec_trace(dec_handle *h, int32_t enable);

/* Copy 4 stamps per kernel for the first n_kernels kernels of the step
 * (order as in dec_launch_kernel) into out[4 * n_kernels] (host). */
int dec_trace_read(dec_handle *h, uint64_t *out, size_t n_kernels);

/* Test hook for the bounded wait: enqueue a kernel that busies one SM for
 * about `microseconds` (clamped to [0, 2000000]) and then ends by itself. */
int dec_debug_busy(dec_handle *h, int64_t microseconds);

/* Test hook: change the wait bound of an existing handle (ms, > 0). */
int dec_set_timeout(dec_handle *h, int64_t wait_timeout_ms);

/* Test hook for the in-kernel bounded waits of the persistent step ("Execution",
 * section "Failure handling": every wait is bounded, and a wait that gives up
 * is a typed error rather than a hang).  Takes effect from the next launch:
 *   grid_polls  polls of a wait on other CTAs (phase counters, attention split
 *               groups) before it gives up; 0: the default (2^22)
 *   ring_polls  polls of a wait on a shared-memory ring stage (a copy landing,
 *               a slot freed) before it gives up; 0: the default (2^22)
 *   hold_phase  phase index whose grid-wide wait target is raised by one, so
 *               that wait cannot complete and gives up after grid_polls
 *               (phases: 0 embedding, 1 + 5l + {0 QKV, 1 attention, 2 O-proj,
 *               3 gate/up, 4 down} of layer l, 5L + 1 head); -1: none
 *   drop_stage  ring stage index (counted over the whole step) that CTA 0's
 *               producer never issues, so its consumers give up after
 *               ring_polls; -1: none
 * A wait that gives up sets DEC_FAULT_WAIT in the error word; the kernel then
 * skips the remaining work, waits (bounded) for its own copies in flight and
 * exits; the step returns DEC_E_DEVICE_FAULT and the handle needs
 * dec_reset_state.  (0, 0, -1, -1) restores the defaults.  DEC_E_STATE unless
 * the capture uses DEC_STRATEGY_PERSISTENT; DEC_E_INVALID for hold_phase or
 * drop_stage below -1. */
int dec_debug_wait(dec_handle *h, uint32_t grid_polls, uint32_t ring_polls, int32_t hold_phase, int32_t drop_stage);

const char *dec_last_error(const dec_handle *h);
const char *dec_status_str(int status);

/* Release the handle ("Execution", executor contract: unload): after a
 * bounded wait for its stream, free everything the library allocated (graph,
 * library-owned workspace, pinned staging, stream and event).  Borrowed
 * weights and a caller workspace are not touched.  A poisoned handle frees
 * only host state and leaks the device memory that pending work could
 * reference ("Execution", section "Failure handling").  DEC_E_INVALID for
 * NULL; the handle is invalid afterwards whatever the status. */
int dec_destroy(dec_handle *h);

#ifdef __cplusplus
}
#endif
#endif /* GRAPHDEC_H */
