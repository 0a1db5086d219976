// kv8_step.cu -- a decode step's new q, K and V for a capture with an e4m3 K/V
// store: RoPE of every row's q and k at Pos, and k, v into the row's store at
// the step's position (contiguous) or WriteMap slot (paged), by the rules of
// dec_kv8_append.
//
// Several rows may write into the same block (a prompt's chunk steps as rows of
// one sequence), at any positions in any order; its scale is one, so the first
// of those rows' CTAs writes for all of them, as one append: the largest of all
// their values gives the exponent, and what the block holds below the last of
// their positions is rounded again if that grew.  Of rows that write the same
// position the last one counts.  One CTA for each row and K or V head, and for
// each query head; a thread for each dim.  A few kilobytes: what it costs is
// its launch and two dependent trips to memory.
#include <limits.h>
#include "kv8.cuh"

namespace gd {

namespace {

constexpr int KV8_STEP_ROWS = 8;   // of a step, at most

// grid (2 * Hkv + Hq, R), HD threads
template <int HD>
__global__ void __launch_bounds__(HD) k_kv8_step(const Kv8Step p) {
    __shared__ float tops[HD / 32];
    pdl_wait();
    const Kv8Cache& c = p.c;
    const int r = blockIdx.y, d = threadIdx.x, H2 = HD / 2;
    const int head = blockIdx.x;   // K heads, V heads, query heads
    auto value = [&](int row, int at, bool turn) {   // dim d of the head at `at` of the row's q | k | v
        const float* x = p.qkv + (size_t)row * p.qkv_stride + at;
        if (!turn) return x[d];
        const int pos = min(max(p.pos[row], 0), p.cap - 1);   // out of range: flagged by the embedding and the attention
        const float2 cs = p.rope[(size_t)pos * H2 + (d < H2 ? d : d - H2)];
        return d < H2 ? x[d] * cs.x - x[d + H2] * cs.y : x[d - H2] * cs.y + x[d] * cs.x;
    };
    if (head >= 2 * c.Hkv) {
        const int hq = head - 2 * c.Hkv;
        p.q_out[((size_t)r * p.Hq + hq) * HD + d] = value(r, hq * HD, true);
        pdl_trigger();
        return;
    }
    const bool is_v = head >= c.Hkv;
    const int h = is_v ? head - c.Hkv : head;
    // where a row writes, in positions of the pool; -1: nowhere
    auto target = [&](int row) -> long long {
        if (!p.write_map) {
            const int pos = p.pos[row];
            return pos < 0 || pos >= p.cap ? -1ll : (long long)row * c.page + pos;
        }
        const int slot = p.write_map[row];
        return slot < 0 || slot >= (long long)c.num_pages * c.page ? -1ll : (long long)slot;
    };
    long long to[KV8_STEP_ROWS];
#pragma unroll
    for (int i = 0; i < KV8_STEP_ROWS; ++i) to[i] = i < p.R ? target(i) : -1ll;
    const long long mine = target(r);
    if (mine < 0) {
        if (d == 0 && p.write_map) atomicOr(p.err, FAULT_WRITE_MAP);
        pdl_trigger();
        return;
    }
    const long long block = mine >> c.block_log2;
    bool own = true;
#pragma unroll
    for (int i = 0; i < KV8_STEP_ROWS; ++i) own &= !(i < r && to[i] >= 0 && to[i] >> c.block_log2 == block);
    if (!own) {   // an earlier row's CTA writes for this one
        pdl_trigger();
        return;
    }
    // the block's first byte and its scale
    const long long page = mine / c.page;
    const int first = (int)(mine % c.page) >> c.block_log2 << c.block_log2;
    uint8_t* store = (is_v ? c.v : c.k) + (((size_t)page * c.Hkv + h) * c.page + first) * HD;
    uint8_t* scale = (is_v ? c.vs : c.ks) + ((size_t)page * c.Hkv + h) * (c.page >> c.block_log2) + (first >> c.block_log2);
    const int had = (int)*scale - 127;
    float x[KV8_STEP_ROWS], top = 0.f;
    int at[KV8_STEP_ROWS], last = 0;   // position in the block, -1: not a row of this block
    unsigned long long written = 0;    // a block has at most 64 positions
#pragma unroll
    for (int i = 0; i < KV8_STEP_ROWS; ++i) {
        at[i] = to[i] >= 0 && to[i] >> c.block_log2 == block ? (int)(to[i] & (c.block - 1)) : -1;
#pragma unroll
        for (int j = i + 1; j < KV8_STEP_ROWS; ++j)
            if (to[j] == to[i]) at[i] = -1;
        if (at[i] < 0) continue;
        x[i] = value(i, is_v ? (p.Hq + c.Hkv + h) * HD : (p.Hq + h) * HD, !is_v);
        if (fabsf(x[i]) <= 3.402823466e38f) top = fmaxf(top, fabsf(x[i]));
        written |= 1ull << at[i];
        last = max(last, at[i]);
    }
    top = warp_max(top);
    if ((d & 31) == 0) tops[d >> 5] = top;
    __syncthreads();   // and every thread has read the old exponent
    top = tops[0];
#pragma unroll
    for (int w = 1; w < HD / 32; ++w) top = fmaxf(top, tops[w]);
    const unsigned long long held = ((1ull << last) - 1) & ~written;   // earlier positions in the block
    int e = kv8_exponent(top);
    if (held) e = max(e, had);
    if (held && e > had) {
        const float f = pow2i(max(had - e, -60));
        for (unsigned long long m = held; m; m &= m - 1) {   // each thread its own dim: no other thread's bytes
            uint8_t* y8 = store + (size_t)(__ffsll((long long)m) - 1) * HD + d;
            float y[4];
            e4m3x4_to_f32(*y8, y);
            *y8 = (uint8_t)f32_to_e4m3x4(y[0] * f, 0.f, 0.f, 0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < KV8_STEP_ROWS; ++i) {
        if (at[i] < 0) continue;
        float y = x[i] * pow2i(-min(e, 126));
        if (!(fabsf(y) <= 448.f)) y = __int_as_float(0x7FFFFFFF);
        store[(size_t)at[i] * HD + d] = (uint8_t)f32_to_e4m3x4(y, 0.f, 0.f, 0.f);
    }
    if (d == 0) *scale = (uint8_t)(e + 127);
    pdl_trigger();
}

}  // namespace

cudaError_t kv8_step_launch(const Kv8Step& p, cudaStream_t s, bool pdl) {
    if (p.R > KV8_STEP_ROWS || p.c.block > 64) return cudaErrorInvalidValue;   // a capture has neither
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * p.c.Hkv + p.Hq, p.R);
    cfg.blockDim = dim3(p.c.hd);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return p.c.hd == 128 ? cudaLaunchKernelEx(&cfg, k_kv8_step<128>, p) : cudaLaunchKernelEx(&cfg, k_kv8_step<64>, p);
}

cudaError_t attn_kv8_launch(const AttnPlan& a, cudaStream_t s, bool pdl) {
    const AttnParams& p = a.p;
    Kv8Step st{a.cache, p.qkv, p.qkv_stride, p.Hq, p.R, p.cap, p.pos, a.paged ? p.write_map : nullptr, p.rope, a.q_rot, p.err};
    cudaError_t e = kv8_step_launch(st, s, pdl);
    if (e != cudaSuccess) return e;
    Kv8Attend t{};
    t.c = a.cache;
    t.b = Kv8Batch{nullptr, p.pos, p.R, 1, p.err, 1};
    t.q = a.q_rot;
    t.out = p.out;
    t.q_stride = t.out_stride = (long long)p.Hq * p.hd;
    t.dtype = W_F32;
    t.heads(p.Hq);
    t.window = a.window ? a.window : INT_MAX;
    t.sinks = a.window ? a.sinks : 0;
    t.scale = p.scale;
    t.counters = a.kv8_counters;
    t.ws = a.kv8_ws;
    return kv8_decode_launch(t, a.num_sms, s);
}

}  // namespace gd
