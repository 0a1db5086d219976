// internal.h -- launch interface between the engine (engine.cu) and the
// kernel translation units.  Host-side only; no torch types anywhere.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <atomic>
#include "graphdec.h"

namespace gd {

// Raise a kernel's dynamic shared-memory cap to the device's opt-in limit
// minus its static shared memory.  The cap is per function and shared by every
// handle in the process, so it is raised once to the limit rather than set to
// one plan's size (a smaller later value would break an earlier plan).
inline cudaError_t raise_smem_cap(const void* fn) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, fn);
    if (e != cudaSuccess) return e;
    int dev = 0, optin = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - (int)fa.sharedSizeBytes);
}

enum WType { W_F32 = 0, W_BF16 = 1 };

// ---------------- fused norm + GEMV ----------------
// out[r, n] (=|+=) sum_k W[n, k] * a[r, k] for the rows n of up to three
// weight segments stacked in one output index space (e.g. Wq;Wk;Wv).
// The activation a is built in shared memory by the prologue:
//   PRO_PLAIN   a = act
//   PRO_RMSNORM a = act / sqrt(mean(act^2) + eps) * gain
//   PRO_SWIGLU  a = silu(act[:, :K]) * act[:, K:2K]
enum Prologue { PRO_PLAIN = 0, PRO_RMSNORM = 1, PRO_SWIGLU = 2 };
// Epilogue: store, add into out (residual), or store logits + greedy argmax.
// EPI_SWIGLU (tensor-core GEMV only): segments 0 and 1 are gate and up with the
// same row count F, and out[r, n] = silu(gate_n . a_r) * (up_n . a_r), n < F.
enum Epilogue { EPI_STORE = 0, EPI_ADD = 1, EPI_LOGITS = 2, EPI_SWIGLU = 3 };

struct GemvParams {
    const void* w[3];
    int seg_rows[3];
    int N;                 // total output rows
    int K;                 // reduction length
    int R;                 // activation rows in use (<= the kernel's NR)
    const float* act;      // [R, act_stride] fp32
    int act_stride;
    const void* gain;      // [K] in the weight dtype (PRO_RMSNORM)
    float eps;
    float* out;            // [R, out_stride] fp32
    int out_stride;
    unsigned long long* amax;  // [R] argmax keys (EPI_LOGITS)
    unsigned* nonfinite;       // [R] flags (EPI_LOGITS)
    unsigned* err;             // error word (FAULT_WAIT)
    int rps;                   // weight rows per ring stage (tensor-core GEMV: tiles per row group)
    int stages;                // ring stages
    int tc_bh;                 // box-streamed tensor-core GEMV: rows per box (row group)
    int tc_seg_ranges[3];      // box-streamed tensor-core GEMV: row ranges per segment
    int tc_ws;                 // tensor-core GEMV: weight columns per stage
    int tc_ks;                 // tensor-core GEMV: K splits (CTAs per row range)
    float* tc_part;            // tensor-core GEMV, tc_ks > 1: partial sums [ks][R][N or 2F] + [ks][ranges][8] sums of squares
    size_t tc_part_cap;        // floats available at tc_part
    unsigned* tc_cnt;          // tensor-core GEMV, tc_ks > 1: arrivals per row range (zero between launches)
    unsigned long long* trace; // trace buffer or null
    int trace_id;
};

struct W4Gemv;
struct GemvPlan {
    const W4Gemv* w4 = nullptr;   // matrices in 4 bits: the plan that runs (w4_gemv.cu), owned by the engine; p still says
                                  // the shape, and nothing else below is used
    int wtype, pro, epi, nr, cpl;
    int tc;                // 1: tensor-core GEMV (gemv_tc.cu), 2: box-streamed tensor-core GEMV (gemv_tma.cu)
    alignas(64) unsigned char tma_maps[3 * 128];   // tc == 2: one TMA tensor map per weight segment
    int grid, block;
    size_t smem;
    GemvParams p;
};

// Fill plan->grid/block/smem/nr/cpl and p.rps/p.stages for the given shape.
cudaError_t gemv_plan(GemvPlan* plan, int num_sms);
// Scratch of the tensor-core GEMV for rows x (K -> N) (paired: N = 2F): floats
// of split partials, and the arrival counters (words), for any device.
size_t gemv_tc_part_floats(int R, int K, int N, bool paired);
// the same for the box-streamed tensor-core GEMV (it splits K up to 16 ways)
size_t gemv_box_part_floats(int R, int K, int N);
constexpr size_t GEMV_TC_CNT_WORDS = 1024;
cudaError_t gemv_launch(const GemvPlan& plan, cudaStream_t s, bool pdl);

// ---------------- the 8-bit K/V cache (kv8*.cu) ----------------
constexpr int KV8_MAX_ROWS = 1024;
// what a kernel needs to be told once on each device (a race only tells it twice)
struct OncePerDevice {
    std::atomic<unsigned long long> done{0};
    template <typename F>
    cudaError_t run(F f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        if ((e = f()) == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};
// n / d for 0 <= n < 2^31 without a division: mul = ceil(2^(31 + shift) / d), shift = ceil(log2 d)
struct FastDiv {
    unsigned d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(unsigned d_) : d(d_), shift(0) {
        while ((1ull << shift) < d) ++shift;
        mul = (unsigned)(((1ull << (31 + shift)) + d - 1) / d);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int of(int n) const { return (int)(__umulhi((unsigned)n << 1, mul) >> shift); }
#endif
};
struct Kv8Cache {              // a dec_kv8_cache that passed its checks
    uint8_t *k, *v;            // [num_pages, Hkv, page, hd] e4m3
    uint8_t *ks, *vs;          // [num_pages, Hkv, page / block] exponent + 127
    const int* pages;          // [rows, ppr] or null: row r owns pages r * ppr ..
    int rows, ppr, page, num_pages, Hkv, hd, block, block_log2;
    FastDiv by_page;
};
inline int kv8_log2(int block) { return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7; }
struct Kv8Batch {
    const int* q_start;        // [rows + 1] or null: one token a row
    const int* kv_len;         // [rows], or null: one row of len_add positions with all tokens
    int total, max_new;
    unsigned* err;
    int len_add;               // added to kv_len: 1 where it is the position of a row's one token
};
struct Kv8Append {
    Kv8Cache c;
    Kv8Batch b;
    const void *k, *v;         // [total, Hkv, hd], token strides below (elements)
    long long k_stride, v_stride;
    int dtype;                 // W_F32 / W_BF16
};
struct Kv8Attend {
    Kv8Cache c;
    Kv8Batch b;
    const void* q;             // [total, Hq, hd]
    void* out;                 // [total, Hq, hd]
    long long q_stride, out_stride;
    int dtype, Hq;
    int G;                     // query heads of a K/V head
    FastDiv by_group;
    void heads(int n) {
        Hq = n;
        G = n / c.Hkv;
        by_group = FastDiv((unsigned)G);
    }
    int window, sinks;         // window INT_MAX: every position up to the token's own
    int skip, take;            // kv8_decode: a launch's tokens of each row, [skip, skip + take); take 0: all
    float scale;
    int* counters;             // [rows, Hkv], zero between calls
    float* ws;                 // kv8_decode_floats() or kv8_prompt_floats() floats
};
// a decode step's q, K and V (kv8_step.cu)
struct Kv8Step {
    Kv8Cache c;
    const float* qkv;          // [R, qkv_stride]: q, k, v of every row, before RoPE
    int qkv_stride, Hq, R, cap;
    const int* pos;            // [R] Pos slot
    const int* write_map;      // [R] WriteMap slot (paged) or null
    const float2* rope;        // [cap, hd / 2]
    float* q_out;              // [R, Hq * hd]: q after RoPE
    unsigned* err;
};
cudaError_t kv8_step_launch(const Kv8Step& p, cudaStream_t s, bool pdl);
cudaError_t kv8_append_launch(const Kv8Append& p, cudaStream_t s);
// up to 16 query rows (tokens x query heads of a K/V head) of a sequence, or a few times as many (kv8_decode.cu)
bool kv8_decode_takes(const Kv8Attend& p, int num_sms);
cudaError_t kv8_decode_launch(const Kv8Attend& p, int num_sms, cudaStream_t s);
size_t kv8_decode_floats(const Kv8Attend& p, int num_sms);   // of workspace
// any number of query rows (kv8_prompt.cu)
cudaError_t kv8_prompt_launch(const Kv8Attend& p, int num_sms, cudaStream_t s);
size_t kv8_prompt_floats(const Kv8Attend& p, int num_sms);

// ---------------- 4-bit weights (w4*.cu) ----------------
struct W4Matrix {              // a dec_w4_weight that passed its checks
    const void* codes;         // [n, k / 2]
    const void* scales;        // [n, k / group] bf16
    int n, k, group;
};
// a weight's checks: DEC_OK, or a status and the calling thread's message
int w4_check(const char* what, const dec_w4_weight* w, W4Matrix* out);
cudaError_t w4_quantize_launch(const W4Matrix& w, const void* src, long long stride, bool f32, int num_sms, cudaStream_t s);
cudaError_t w4_values_launch(const W4Matrix& w, void* dst, long long stride, bool f32, int num_sms, cudaStream_t s);
// out[t, n] = residual[t, n] + sum_k W[n, k] a[t, k] over up to three matrices of one k and group, stacked; with glu, over a
// gate and an up matrix of one shape, out[t, n] = act(gate[t, n]) * up[t, n].  a = x, or RMSNorm(x) with a gain
struct W4Call {
    W4Matrix w[3];
    int nw;
    bool glu;
    int act;                   // DEC_ACT_*
    int tokens;
    const void* x;             // [tokens, k]
    const void* gain;          // [k] or null: no norm
    const void* residual;      // [tokens, n] or null
    void* out;                 // [tokens, n]
    long long x_stride, residual_stride, out_stride;   // elements
    bool x_f32, gain_f32, out_f32;                      // else bf16; the residual has out's type
    float eps;
    unsigned* err;
    int n() const { return glu ? w[0].n : w[0].n + (nw > 1 ? w[1].n : 0) + (nw > 2 ? w[2].n : 0); }
    int k() const { return w[0].k; }
    int group() const { return w[0].group; }
    // fp16 parts of an activation, for few tokens and many alike.  A normed bf16 one is a product with a gain, of more than
    // the 11 bits of one part: with one, results are off by 2e-4 of the whole, and a tenth of bf16 results are a step off.
    // Two cost 28 us in place of 22 (40 tokens, 6144 x 4096) and 2020 in place of 899 (4095 tokens, gate and up 14336 x 4096)
    int parts() const { return x_f32 || gain ? 2 : 1; }
};
struct W4Gemv {                // how w4_gemv.cu runs a call of few tokens
    W4Call c;
    int block;                 // tokens of a CTA
    int wk;                    // warps along k
    int ks;                    // CTAs along k, a cluster
    int grid, rows;            // CTAs along n, output rows of each (the last may have fewer)
    int stages;                // ring steps
    int bufs;                  // buffers of the cross-warp sums
    size_t smem;
    unsigned long long* amax;  // logits of a decode step: [tokens] argmax keys, or null
    unsigned* nonfinite;       // [tokens]
    unsigned long long* trace;
    int trace_id;
};
int w4_clusters(int ks, int num_sms);   // clusters of ks CTAs, one CTA an SM, that run at a time
cudaError_t w4_gemv_plan(W4Gemv* g, int num_sms);
cudaError_t w4_gemv_launch(const W4Gemv& g, cudaStream_t s, bool pdl);
struct W4Gemm {                // how w4_gemm.cu runs a call of many tokens
    W4Call c;                  // nw == 1, or glu
    int parts;                 // fp16 parts of an activation: c.parts(), or two because the sums are to be folded
    int nt;                    // tokens of an accumulator
    bool wide;                 // one row tile and two blocks of nt tokens a CTA, or two row tiles and one block
    int ks;                    // CTAs along k, a cluster
    int kp, steps;             // columns rounded up to 64; steps of 128
    void* ws;                  // w4_gemm_bytes()
};
cudaError_t w4_gemm_plan(W4Gemm* g, int num_sms);
size_t w4_gemm_bytes(const W4Gemm& g);
cudaError_t w4_gemm_launch(const W4Gemm& g, cudaStream_t s);

// ---------------- split-KV masked decode attention ----------------
struct AttnParams {
    const float* qkv;      // [R, qkv_stride]: q [Hq*hd], k [Hkv*hd], v [Hkv*hd] (fp32, pre-RoPE)
    int qkv_stride;
    void* Kc;              // this layer's K store (layout per `paged`)
    void* Vc;
    const int* pos;        // [R] slot
    const int* slot_map;   // [R, pages_per_row] slot (paged)
    const int* write_map;  // [R] slot (paged)
    const float2* rope;    // [cap, hd/2] (cos, sin)
    int cap, R, Hq, Hkv, hd;
    int split_len, nsplit;
    int stages;            // ring stages
    int page_size, pages_per_row, num_pages;
    float* part;           // [R, Hq, nsplit, hd + 2] partial (m, l, o)
    unsigned* counters;    // [R, Hkv] split-completion counters (zero between steps)
    float* out;            // [R, Hq * hd]
    unsigned* err;
    int kv_prewritten;     // 1: every row's new k, v are already in the store (k_kv_write ran)
    int pos_bound;         // 1: a split loads no K/V tile after the one holding pos (DEC_SWEEP_POS)
    float scale;
    unsigned long long* trace;
    int trace_id;
};

struct AttnPlan {
    int kvtype;   // W_F32 / W_BF16
    bool paged;
    int group;    // Hq / Hkv
    dim3 grid;
    int block;
    size_t smem;
    AttnParams p;
    bool mma = false;              // tensor-core kernel (attn_mma.cu)
    void* mma_params = nullptr;    // its parameter block (tensor maps + p), owned by the plan
    bool prewrite = false;         // launch k_kv_write before the attention (p.kv_prewritten = 1)
    bool kv8 = false;              // e4m3 store: kv8_step.cu, then kv8_decode.cu, with what stands below
    Kv8Cache cache{};
    float* q_rot = nullptr;        // [R, Hq * hd]
    int* kv8_counters = nullptr;
    float* kv8_ws = nullptr;
    int window = 0, sinks = 0, num_sms = 0;
};

// RoPE of every row's k at Pos, rounding and store of k, v (bf16 store) at the
// row's position or WriteMap slot, before the attention of any row reads them
cudaError_t kv_write_launch(const AttnPlan& plan, cudaStream_t s, bool pdl);

// the attention of an e4m3 store: two launches
cudaError_t attn_kv8_launch(const AttnPlan& plan, cudaStream_t s, bool pdl);
// choose split_len / nsplit; returns cudaErrorInvalidValue for unsupported head_dim / group
cudaError_t attn_plan(AttnPlan* plan, int num_sms);
cudaError_t attn_launch(const AttnPlan& plan, cudaStream_t s, bool pdl);
size_t attn_part_floats(int R, int Hq, int hd, int nsplit);

// tensor-core variant for bf16 K/V (head_dim 64 or 128)
bool attn_mma_supported(int kvtype, int hd, int G, bool paged, int page_size);
cudaError_t attn_mma_plan(AttnPlan* plan, int num_sms);
cudaError_t attn_mma_launch(const AttnPlan& plan, cudaStream_t s, bool pdl);
void attn_mma_release(AttnPlan& plan);

// ---------------- embedding gather + per-step resets ----------------
struct EmbedParams {
    const void* E;         // [V, d] weight dtype
    const int* tok;        // [R]
    const int* pos;        // [R]
    int R, V, d, cap;
    float* x;              // [R, d]
    unsigned* err;
    unsigned long long* amax;
    unsigned* nonfinite;
    unsigned long long* trace;
    int trace_id;
};
cudaError_t embed_launch(int wtype, const EmbedParams& p, cudaStream_t s);

// ---------------- sampling suffix ----------------
struct SamplerSlot {                 // device copy of dec_sampler (same field order)
    float temperature;
    int top_k;
    float top_p;
    float min_p;
    unsigned long long seed;
    int n_logprobs;
    int reserved;
};
struct SampleParams {
    const float* logits;             // [R, V]
    int V, R;
    const unsigned long long* amax;  // [R] greedy keys
    const int* pos;                  // [R] Pos slot (the uniform's counter)
    const SamplerSlot* cfg;          // parameter slot
    int* sampled;                    // [R] picks
    int* lp_ids;                     // [R, DEC_LOGPROBS_MAX]
    float* lp_vals;                  // [R, DEC_LOGPROBS_MAX]
};
cudaError_t sample_launch(const SampleParams& p, cudaStream_t s);

// ---------------- chained greedy steps ----------------
struct ChainParams {
    int* tok;                        // [R] Token slot
    int* pos;                        // [R] Pos slot
    int* wm;                         // [R] WriteMap slot (paged)
    const int* slot_map;             // [R, ppr] SlotMap (paged) or null
    int R, V, cap, ppr, page;
    const unsigned long long* amax;  // [R] greedy keys of the step just run
    const unsigned* nonfinite;       // [R]
    unsigned* err;                   // the step's error word
    unsigned* chain_err;             // sticky over the chain
    const int* sampled;              // [R] sampled ids, or null: greedy keys
    int* counter;                    // steps recorded so far
    int* ids;                        // [max_steps, R] history
    int* nf;                         // [max_steps, R] history
    int max_steps;
};
cudaError_t chain_advance_launch(const ChainParams& p, cudaStream_t s);

// a kernel that spins for about `ns` nanoseconds on one SM, then returns
cudaError_t busy_launch(long long ns, cudaStream_t s);

// ---------------- the whole step as one persistent kernel ----------------
struct PersistParams {
    int L, d, F, V, Hq, Hkv, hd, R, cap;
    int paged, page, pages_per_row, num_pages;
    float eps, scale;
    const void* const* lw;     // [L * 9] device table: attn_norm, q, k, v, o, ffn_norm, gate, up, down
    const void* embed;
    const void* final_norm;
    const void* lm_head;
    float* x;
    float* qkv;
    float* attn;
    float* gu;
    float* logits;
    float* part;
    unsigned* counters;        // [R * Hkv] split completion
    const int* slots;          // tokens [R], pos [R], write map [R]
    const int* slot_map;
    const float2* rope;
    void* const* kv;           // [L * 2] device table: K, V store of each layer
    const void* tmaps;         // [L][K|V][2] tensor maps in device memory (64-byte aligned)
    unsigned* err;
    unsigned long long* amax;
    unsigned* nonfinite;
    unsigned* bar;             // [5L + 5]: per-phase arrivals, exit counter, abort word, head block counter
    unsigned long long* trace;
    int split_len, nsplit;
    int rps_d, rps_f;          // weight rows per ring stage for K = d and K = F
    const unsigned* dbg;       // [4] wait bounds and test hooks: grid-wait polls, ring-wait polls (0: defaults),
                               // phase whose grid-wait target is raised by one + 1, stage CTA 0 never issues + 1
                               // (0: none); 16-byte aligned
};

struct PersistPlan {
    PersistParams p;
    int grid = 0, block = 0;
    size_t smem = 0;
    const void* fn = nullptr;
};

// fills split_len / nsplit / rps_* and the launch shape; cudaErrorNotSupported
// when this shape has no persistent kernel
cudaError_t persist_plan(PersistPlan* plan, int num_sms);
size_t persist_tmap_bytes(int n_layers);
// host images of the layer tensor maps (written to the device table by the caller)
cudaError_t persist_tmaps(const PersistParams& p, void* const* kv, void* host_out);
cudaError_t persist_launch(const PersistPlan& plan, cudaStream_t s);

// ---------------- multi-token prefill of one sequence (prefill.cu) ----------------
struct PrefillArgs {
    int L, d, Hq, Hkv, hd, F, cap;
    float eps;
    const void* embed;          // [V, d] bf16
    const void* const* lw;      // host array [L * 9] of device pointers: attn_norm, q, k, v, o, ffn_norm, gate, up, down
    void* const* K;             // host array [L] of device pointers: K store of each layer
    void* const* V;             // host array [L]: V store
    bool kv8;                   // e4m3 store, with scales and perhaps a window; else bf16
    void* const *KS, *const *VS;   // host arrays [L]: scales of each layer
    int block, window, sinks;
    bool paged;
    int page, ppr;              // paged: tokens per page, pages per sequence
    int rows, num_pages;        // contiguous: the capture's rows; paged: the pool's pages
    const float2* rope;         // device [cap, hd / 2]
    unsigned* err;              // device error word
};
struct PrefillState;
// whether this shape has a block prefill (bf16 weights and K/V are the caller's check)
bool prefill_supported(const PrefillArgs& a);
// device buffers and tensor maps of the block prefill (cudaMalloc; freed by prefill_free)
cudaError_t prefill_create(const PrefillArgs& a, int num_sms, PrefillState** out);
void prefill_free(PrefillState* s);
// n tokens (host) at positions pos0 .. pos0 + n - 1 of sequence `row` (contiguous
// K/V) or of the sequence on `pages` (host, paged K/V): every layer's K/V of those
// positions written; the last token's hidden state (fp32 [d]) to x_last (device)
cudaError_t prefill_run(PrefillState* s, const int* tokens, int n, int pos0, int row, const int* pages, float* x_last,
                        cudaStream_t st);

}  // namespace gd

struct dec_handle;
namespace gd {
// engine services for other translation units of the library
int engine_run_attention(dec_handle* h, int32_t layer, const float* qkv, const int32_t* pos, float* out, float* part,
                         unsigned* counters);
void engine_attention_scratch(const dec_handle* h, size_t* part_floats, size_t* counters);
int engine_gate(dec_handle* h);
int engine_fail(dec_handle* h, int code, const char* msg);
int engine_device(const dec_handle* h);
// the message that dec_last_error(NULL) gives on this thread
void set_call_message(const char* msg);
const char* call_message();

}  // namespace gd
