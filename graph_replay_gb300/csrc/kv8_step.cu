// kv8_step.cu -- a decode step's new q, K and V for a capture with an e4m3 K/V
// store: RoPE of every row's q and k at Pos, and k, v into the row's store at
// the step's position (contiguous) or WriteMap slot (paged), by the rules of
// dec_kv8_append.
//
// Several rows may write into the same block (a prompt's chunk steps as rows of
// one sequence); its scale is one, so the first of those rows' CTAs writes for
// all of them, in row order.  One CTA for each row and K or V head, and for
// each query head; a thread for each dim.  A few kilobytes: what it costs is
// its launch and two dependent trips to memory.
#include <limits.h>
#include "kv8.cuh"

namespace gd {

namespace {

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
    const long long mine = target(r);
    if (mine < 0) {
        if (d == 0 && p.write_map) atomicOr(p.err, FAULT_WRITE_MAP);
        pdl_trigger();
        return;
    }
    const long long block = mine >> c.block_log2;
    for (int row = 0; row < r; ++row) {
        const long long t = target(row);
        if (t >= 0 && t >> c.block_log2 == block) {   // that row's CTA writes for this one
            pdl_trigger();
            return;
        }
    }
    // the block's first byte and its scale
    const long long page = mine / c.page;
    const int first = (int)(mine % c.page) >> c.block_log2 << c.block_log2;
    uint8_t* store = (is_v ? c.v : c.k) + (((size_t)page * c.Hkv + h) * c.page + first) * HD;
    uint8_t* scale = (is_v ? c.vs : c.ks) + ((size_t)page * c.Hkv + h) * (c.page >> c.block_log2) + (first >> c.block_log2);
    int had = (int)*scale - 127;
    for (int row = r; row < p.R; ++row) {
        const long long t = target(row);
        if (t < 0 || t >> c.block_log2 != block) continue;
        const int held = (int)(t & (c.block - 1));   // earlier positions in the block
        float x = value(row, is_v ? (p.Hq + c.Hkv + h) * HD : (p.Hq + h) * HD, !is_v);
        float top = warp_max(fabsf(x) <= 3.402823466e38f ? fabsf(x) : 0.f);
        __syncthreads();   // the last row's maxima have been read
        if ((d & 31) == 0) tops[d >> 5] = top;
        __syncthreads();
        top = tops[0];
#pragma unroll
        for (int w = 1; w < HD / 32; ++w) top = fmaxf(top, tops[w]);
        int e = kv8_exponent(top);
        if (held) e = max(e, had);
        x *= pow2i(-min(e, 126));
        if (!(fabsf(x) <= 448.f)) x = __int_as_float(0x7FFFFFFF);
        store[(size_t)held * HD + d] = (uint8_t)f32_to_e4m3x4(x, 0.f, 0.f, 0.f);
        if (held && e > had) {
            const float f = pow2i(max(had - e, -60));
            for (int j = 0; j < held; ++j) {   // each thread its own dim: no other thread's bytes
                float y[4];
                e4m3x4_to_f32(store[(size_t)j * HD + d], y);
                store[(size_t)j * HD + d] = (uint8_t)f32_to_e4m3x4(y[0] * f, 0.f, 0.f, 0.f);
            }
        }
        had = e;
    }
    if (d == 0) *scale = (uint8_t)(had + 127);
    pdl_trigger();
}

}  // namespace

cudaError_t kv8_step_launch(const Kv8Step& p, cudaStream_t s, bool pdl) {
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
