// w4_gemv.cuh -- the products of a few tokens with 4-bit weights (mma.sync, sm_103a).
//
// out[t, n] = sum_k W[n, k] a[t, k] reads each weight once for all tokens, so it is
// bound by the bytes of the codes: at the card's rate an SM has to turn about 45
// codes a clock into products.  One FMA and one conversion a weight and token would
// already be too many for the CUDA cores; here a 16 x 16 tile of codes is the A
// operand of mma.sync m16n8k16 (about one instruction a code to unpack, w4.cuh) and
// the tokens are the 8 columns of B:
//   * codes enter as exact fp16 integers; a group's products are summed in the
//     tensor core over at most 128 columns and then multiplied by the group's scale
//     and added to an fp32 sum, so scales cost 1/16 of an FMA a weight and no
//     rounding of a scaled weight happens;
//   * activations enter as one or two fp16 parts (w4.cuh) scaled for each block of
//     128 columns, so bf16 and fp32 run the same path.  The columns of B are
//     (token, part) pairs;
//   * which of the 16 columns of an MMA step is which is free, as long as A and B
//     agree: lane (g, t) takes the words that it finds in 16 consecutive bytes of
//     its row, or, where a group is shorter, in two or four places of 64 bytes.
// A CTA (one an SM, sixteen warps) owns a range of output rows; `wk` warps share
// its columns, 128 at a time in turn, and 16 / wk sets of warps take row groups in
// turn (32 rows; a gate/up pair: 16 of each).  Each warp copies its own tiles with
// cp.async into a ring of its own, so the loop has no barriers; a row group ends
// with one barrier and a sum over the warps in their order.
// The activations of a CTA's columns stay in shared memory as B fragments.  Where
// they do not fit, a cluster of `ks` CTAs shares the columns of a row range, and each
// of them adds the sums of a part of the rows from the others' shared memory, in
// order (14336 -> 4096, eight fp32 tokens: 21 us; 31 with the parts' sums in memory and
// a last CTA that adds them).  Results do not depend on scheduling.
//
// Measured in captures, fp32 activations, copies of the weights larger than L2 in turn:
//   one token     128256 x 4096, groups of 64, norm   65.8 us   4.2 TB/s (a copy: 6.8)
//                 gate and up 14336 x 4096, norm      20.6 us   2.9 TB/s
//                 14336 -> 4096, residual             13.5 us   2.2 TB/s
//                 4096 x 4096, residual                6.8 us   1.3 TB/s
//   eight tokens  14336 -> 4096, residual             21.2 us
//                 gate and up 14336 x 4096, groups of 32, norm   38.7 us
// The largest is bound by instructions, not by bytes: about 360 for a step of 4096
// codes and warp, 64 % of the issue slots; the integer and the half-precision pipe, each
// of which takes an instruction every other clock, are busy in turn, and the tensor pipe
// at 23 %.  Eight tokens issue in 54 % (14336 -> 4096) and 61 % (groups of 32) of the slots,
// and wait for results and at the row groups' barriers besides.  The small ones are bound by
// their ends: launch, the copy and conversion of the activations (1 to 6 thousand clocks) and
// the join.
#pragma once
#include "w4.cuh"

namespace gd {

constexpr int WG_WARPS = 16;
constexpr int WG_THREADS = WG_WARPS * 32;
constexpr int WG_STEP = 2048;                  // bytes of a step: two tiles of 16 rows x 128 columns
constexpr int WG_PITCH = 33;                   // of 32 rows' sums of one token
constexpr int WG_MAX_TOKENS = 16;
constexpr int WG_STAGES = 4;                   // steps of a warp's ring at most
// A group's sum is multiplied by its token's factor, up to 2^113, before the scale that may bring it back into fp32's range.  The
// sum is at most 2^25 (128 columns, codes of 8, parts up to 2^15), so with factors 2^11 smaller (exact: a power of two down to
// 2^-137) no product leaves that range unless the result does; the outputs are made 2^11 larger (with the norm's factor)
constexpr float WG_LESS = 0x1p-11f, WG_MORE = 0x1p11f;

// one matrix; a gate and an up matrix; two or three stacked
enum { W4_ONE = 0, W4_GLU = 1, W4_STACK = 2 };

// tokens of a CTA whose columns fill NB blocks of 8
__host__ __device__ constexpr int wg_tokens(int P, int NB) { return NB * 8 / P; }

struct W4GemvArgs {
    const uint8_t* codes[3];
    const __nv_bfloat16* scales[3];
    int end[3];                // rows of segments 0, 0 + 1, all
    int N, K, tokens, block, wk, ks, rows, stages, bufs, act, x_f32, gain_f32, out_f32, pdl;
    const void* x;
    const void* gain;
    const void* residual;
    void* out;
    long long x_stride, residual_stride, out_stride;
    float eps;
    unsigned long long* amax;
    unsigned* nonfinite;
    unsigned long long* trace;
    int trace_id;
};

// d = a b
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// d += a b
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, unsigned bytes) {   // the rest of 16 bytes is zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// shared memory by its 32-bit address; in order with the copies' waits
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait(bool four) {   // with a ring of four steps (or two) the oldest group has landed
    if (four) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// G: columns of a group; P: fp16 parts of an activation; NB: blocks of 8 B columns
template <int G, int P, int NB, int KIND>
__global__ void __launch_bounds__(WG_THREADS, 1) k_w4_gemv(const __grid_constant__ W4GemvArgs p) {
    constexpr bool GLU = KIND == W4_GLU;
    constexpr int NG = 128 / G;                // groups of a step
    constexpr int MT = wg_tokens(P, NB);       // tokens that fit
    constexpr int AC = P == 2 ? 2 : 4;         // sums of a lane, tile and column block
    constexpr int GR = GLU ? 16 : 32;          // output rows of a row group
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float ss_s[WG_WARPS][MT];
    __shared__ unsigned long long best_s[8];
    __shared__ unsigned nonfinite_s[8];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int tok0 = blockIdx.y * p.block, m = min(p.block, p.tokens - tok0);
    const int cols = p.block * P;
    const int q = blockIdx.x % p.ks, ri = blockIdx.x / p.ks;
    const int row0 = ri * p.rows, row1 = min(p.N, row0 + p.rows);
    const int chunks = (p.K + 127) >> 7;                        // 128 columns each
    const int ch0 = (int)((long long)q * chunks / p.ks), ch1 = (int)((long long)(q + 1) * chunks / p.ks);
    const int room = (chunks + p.ks - 1) / p.ks;                // chunks of a CTA at most: a cluster's CTAs lay out memory alike
    const int set = warp / p.wk, sets = WG_WARPS / p.wk, slice = warp % p.wk;
    const int ngroups = (row1 - row0 + GR - 1) / GR;            // row groups of the CTA
    const int iters = (ngroups + sets - 1) / sets;              // of each set
    const int mine = (ch1 - ch0 - slice + p.wk - 1) / p.wk;     // this warp's chunks of a row group (>= 0)

    const int S = p.stages;
    const unsigned ring_bytes = (unsigned)S * WG_STEP;
    unsigned char* xs = smem + (size_t)WG_WARPS * ring_bytes;                // [chunk][cols][4][64 bytes], an odd column's words in pairs exchanged: no bank conflicts
    float* fs = reinterpret_cast<float*>(xs + (size_t)room * cols * 256);   // [chunk][block]: 2^(e - 14 - 11)
    unsigned char* gs = reinterpret_cast<unsigned char*>(fs + ((room * p.block + 3) & ~3));   // [chunk][512]: the gain
    float* red = reinterpret_cast<float*>(gs + (p.gain ? room * 512 : 0));   // [bufs][warp][MT][WG_PITCH]
    float* sums = red + p.bufs * WG_WARPS * MT * WG_PITCH;                   // ks > 1: [1 or 2][block][rows], read by the cluster
    const uint32_t ring_at = smem_u32(smem) + (unsigned)warp * ring_bytes;

    unsigned long long* tr = nullptr;
    if (tid == 0) {
        tr = trace_if_on(p.trace);
        trace_mark(tr, p.trace_id, 0);
    }
    if (tid < 8) {
        best_s[tid] = 0ull;
        nonfinite_s[tid] = 0u;
    }

    // ---- the warp's steps: row groups set, set + sets, ...; in each its chunks; two tiles a step ----
    // where this lane's 16 bytes of row g or g + 8 of a tile go, and where its words are
    const int swz = G == 128 ? 0 : G == 64 ? ((g >> 1) & 1) << 1 : (g >> 1) & 3;
    const uint32_t put = (uint32_t)(g * 64 + ((t ^ swz) << 4));
    // bytes of a row's codes and scales; a matrix has less than 2^32 of either, so a row is a 32-bit offset
    const unsigned cpitch = (unsigned)p.K >> 1, spitch = (unsigned)(p.K / G) * 2u;
    struct Rows {                              // of a row group: rows g, g + 8 of tile 0, then of tile 1
        unsigned c[4], s[4];                   // offsets of their codes and scales
        unsigned live[4];                      // 16 where row i is one of the CTA's, else 0
        unsigned seg;                          // W4_STACK: bits 2i, 2i + 1: the matrix that row i lies in
    };
    auto rows_of = [&](int it, Rows& r) {
        const int base = row0 + (it * sets + set) * GR + g;
        r.seg = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = base + (GLU ? 8 * (i & 1) : 8 * i);
            r.live[i] = at < row1 ? 16u : 0u;
            int n = min(at, row1 - 1);         // scales are read of any row
            if (KIND == W4_STACK) {
                const int sg = (n >= p.end[0]) + (n >= p.end[1]);
                n -= sg == 2 ? p.end[1] : sg == 1 ? p.end[0] : 0;
                r.seg |= (unsigned)sg << (2 * i);
            }
            r.c[i] = (unsigned)n * cpitch;
            r.s[i] = (unsigned)n * spitch;
        }
    };
    // the matrix of row i
    auto codes_of = [&](const Rows& r, int i) -> const uint8_t* {
        if (KIND != W4_STACK) return p.codes[GLU ? i >> 1 : 0];
        const unsigned sg = r.seg >> (2 * i) & 3u;
        return sg == 2 ? p.codes[2] : sg == 1 ? p.codes[1] : p.codes[0];
    };
    auto scale_of = [&](const Rows& r, int i) -> const unsigned char* {
        if (KIND != W4_STACK) return reinterpret_cast<const unsigned char*>(p.scales[GLU ? i >> 1 : 0]);
        const unsigned sg = r.seg >> (2 * i) & 3u;
        return reinterpret_cast<const unsigned char*>(sg == 2 ? p.scales[2] : sg == 1 ? p.scales[1] : p.scales[0]);
    };
    const int steps = mine > 0 ? iters * mine : 0;
    const unsigned hop = (unsigned)p.wk * 64;  // bytes of a row from one of the warp's chunks to its next
    const unsigned a_first = (unsigned)(ch0 + slice) * 64 + 16 * t;
    Rows ahead;                                // of the step that is copied next
    int a_it = 0, a_i = 0, a_left = steps;
    unsigned a_at = a_first, a_slot = 0;       // byte of a row; slot of the ring, in bytes
    if (steps > 0) rows_of(0, ahead);
    auto copy_next = [&]() {
        if (a_left > 0) {
            const unsigned in = G == 128 || a_at < cpitch ? ~0u : 0u;   // (k is a multiple of G)
            const uint32_t dst = ring_at + a_slot + put;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (of rows behind the CTA's last and columns behind the row's nothing is read: zeros)
                cp_async16(dst + (uint32_t)((i >> 1) * 1024 + (i & 1) * 512), codes_of(ahead, i) + (size_t)(ahead.c[i] + a_at),
                           in & ahead.live[i]);
            }
            --a_left;
            a_slot = (a_slot + WG_STEP) & (ring_bytes - 1u);   // four steps or two
            a_at += hop;
            if (++a_i == mine) {
                a_i = 0;
                a_at = a_first;
                if (++a_it < iters) rows_of(a_it, ahead);
            }
        }
        cp_commit();
    };
    // Activations are copied as they are to where their fragments will lie: a token's 128 values take no more room than
    // their parts.  All copies are under way at once
    const int nc = (ch1 - ch0 - warp + WG_WARPS - 1) / WG_WARPS;   // chunks that this warp makes fragments of
    auto copy_x = [&]() {
        const unsigned size = p.x_f32 ? 4u : 2u, row = (unsigned)p.K * size, first = (unsigned)(ch0 + warp) * 128u * size + 16u * lane;
        const unsigned char* src = reinterpret_cast<const unsigned char*>(p.x) + (size_t)tok0 * p.x_stride * size;
        const bool on = p.x_f32 || lane < 16;
        for (int r = 0; r < m; ++r, src += (size_t)p.x_stride * size) {
            uint32_t dst = smem_u32(xs) + (unsigned)(warp * cols + r * P) * 256u + 16u * lane;
            unsigned at = first;
            for (int j = 0; j < nc; ++j, at += WG_WARPS * 128u * size, dst += (unsigned)(WG_WARPS * cols) * 256u)
                if (on) cp_async16(dst, src + at, at < row ? 16u : 0u);
        }
        if (p.gain) {
            const unsigned gsize = p.gain_f32 ? 4u : 2u, grow = (unsigned)p.K * gsize;
            unsigned at = (unsigned)(ch0 + warp) * 128u * gsize + 16u * lane;
            uint32_t dst = smem_u32(gs) + (unsigned)warp * 512u + 16u * lane;
            for (int j = 0; j < nc; ++j, at += WG_WARPS * 128u * gsize, dst += WG_WARPS * 512u)
                if (p.gain_f32 || lane < 16) cp_async16(dst, reinterpret_cast<const unsigned char*>(p.gain) + at, at < grow ? 16u : 0u);
        }
        cp_commit();
    };
    if (!p.pdl) {
        copy_x();
        for (int s = 0; s < S - 1; ++s) copy_next();
    } else {
        for (int s = 0; s < S - 1; ++s) copy_next();   // the weights do not depend on the kernel before
        pdl_wait();
        copy_x();
    }
    if (tid == 0) trace_mark(tr, p.trace_id, 1);

    // ---- activations: each warp makes the fragments of every sixteenth chunk, all warps' are used by all ----
    {
        const int w = lane >> 1;               // word of the chunk that the lane's four columns lie in
        const int bt = G == 128 ? w >> 2 : G == 64 ? (w >> 1) & 3 : w & 3;
        const int bq = G == 128 ? w & 3 : G == 64 ? ((w >> 3) << 1) | (w & 1) : w >> 2;
        const bool odd = lane & 1;
        float ss = 0.f;
        if (p.pdl) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (S == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        auto four = [&](const unsigned char* at, bool f32) {   // this lane's four of 128 values
            if (f32) return *reinterpret_cast<const float4*>(at + 16 * lane);
            const uint2 b = *reinterpret_cast<const uint2*>(at + 8 * lane);
            return make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
        };
        for (int r = 0; r < m; ++r) {
            const unsigned char* go = gs + warp * 512;
            unsigned char* o = xs + (size_t)(warp * cols + r * P) * 256;
            float* fo = fs + warp * p.block + r;
#pragma unroll 1
            for (int j = 0; j < nc; ++j, o += (size_t)WG_WARPS * cols * 256, fo += WG_WARPS * p.block, go += WG_WARPS * 512) {
                float4 x = four(o, p.x_f32);
                if (p.gain) {
                    const float4 gv = four(go, p.gain_f32);
                    ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, fmaf(x.w, x.w, ss))));
                    x.x *= gv.x; x.y *= gv.y; x.z *= gv.z; x.w *= gv.w;
                }
                // (the vote also has every lane's values read before any lane writes over them)
                const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(w4_finite_bits(x.x), w4_finite_bits(x.y)),
                                                                        max(w4_finite_bits(x.z), w4_finite_bits(x.w))));
                __syncwarp();
                const int e = w4_exponent(top);
                const float up = w4_up(e);
                x.x *= up; x.y *= up; x.z *= up; x.w *= up;
#pragma unroll
                for (int part = 0; part < P; ++part) {
                    const uint32_t a01 = w4_pack_half(x.x, x.y), a23 = w4_pack_half(x.z, x.w);
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a01 : a23, 1);
                    const uint32_t lo = odd ? got : a01, hi = odd ? a23 : got;     // columns j and j + 4 of the word
                    const int swap = (r * P + part) & 1;   // of an odd column
                    *reinterpret_cast<uint2*>(o + part * 256 + (bq ^ swap) * 64 + bt * 16 + (odd ? 8 : 0)) =
                        make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
                    if (part + 1 < P) {        // what the part leaves (nothing where it is not finite)
                        const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&a01));
                        const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&a23));
                        x.x -= f01.x; x.y -= f01.y; x.z -= f23.x; x.w -= f23.y;
                        x.x = isfinite(x.x) ? x.x : 0.f; x.y = isfinite(x.y) ? x.y : 0.f;
                        x.z = isfinite(x.z) ? x.z : 0.f; x.w = isfinite(x.w) ? x.w : 0.f;
                    }
                }
                if (lane == 0) *fo = w4_down(e) * WG_LESS;
            }
            if (p.gain) {
                ss = warp_sum(ss);
                if (lane == 0) ss_s[warp][r] = ss;
                ss = 0.f;
            }
        }
        if (p.gain && p.ks > 1) {   // the other CTAs' columns, for the norm: a load of every token at a time
            __syncwarp();
            float s2[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) s2[i] = 0.f;
            for (int c = warp; c < chunks; c += WG_WARPS) {
                const int k = c * 128 + 4 * lane;
                if ((c >= ch0 && c < ch1) || k >= p.K) continue;
                float4 x[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    x[i] = i < m ? w4_load4(p.x, p.x_f32, (size_t)(tok0 + i) * p.x_stride + k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    s2[i] = fmaf(x[i].x, x[i].x, fmaf(x[i].y, x[i].y, fmaf(x[i].z, x[i].z, fmaf(x[i].w, x[i].w, s2[i]))));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float s = warp_sum(s2[i]);
                if (lane == 0 && i < m) ss_s[warp][i] += s;
            }
        }
    }
    // where all warps share the columns, a warp's chunks are those that it made itself
    if (p.wk < WG_WARPS) __syncthreads();
    else __syncwarp();
    pdl_trigger();

    // one output: gate / value v and up u, 2^11 too small and unscaled by the norm; its residual
    float inv = WG_MORE;                       // with that of the norm of token inv_of
    int inv_of = -1;
    auto finish = [&](int r, int n, float v, float u, float res) {
        if (p.gain) {                          // (behind a row group's barrier)
            if (r != inv_of) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < WG_WARPS; ++w) s += ss_s[w][r];
                inv = WG_MORE / sqrtf(s / (float)p.K + p.eps);
                inv_of = r;
            }
        }
        v *= inv;
        u *= inv;
        v = GLU ? w4_glu(p.act, v, u) : v + res;
        w4_store1(p.out, p.out_f32, (size_t)(tok0 + r) * p.out_stride + n, v);
        if (!GLU && p.amax) {
            atomicMax(&best_s[r], argmax_key(v, n));
            if (!isfinite(v)) nonfinite_s[r] = 1u;
        }
    };
    auto residual_of = [&](int r, int n) -> float {
        return !GLU && p.residual ? w4_load1(p.residual, p.out_f32, (size_t)(tok0 + r) * p.residual_stride + n) : 0.f;
    };
    // The joining of a row group's sums: four threads an output, each takes a part of the warps.  A thread's first output is
    // row j_row of set j_set's row group, token j_tok; its next ones are J_NEXT (set, token) pairs further
    constexpr int RG = GLU ? 16 : 32, J_NEXT = WG_THREADS / 4 / RG;
    const int j_row = (tid >> 2) % RG, j_set = (tid >> 2) / RG / m, j_tok = (tid >> 2) / RG - j_set * m;

    // ---- the products ----
    // the scales of the step after this one: of row g in the low half, of row g + 8 in the high half, of group t (one of
    // NG); raw bits
    Rows cur, next;
    // two sets in turn: moving one into the other would wait for the loads
    uint32_t s_even[4] = {0u, 0u, 0u, 0u}, s_odd[4] = {0u, 0u, 0u, 0u};
    const unsigned g_first = 2u * (unsigned)((ch0 + slice) * NG + (NG > 1 ? t % NG : 0)), g_hop = 2u * (unsigned)(p.wk * NG);
    auto scales_of = [&](const Rows& r, unsigned at, uint32_t (&o)[4]) {
        at = min(at, spitch - 2u);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __ldg(reinterpret_cast<const unsigned short*>(scale_of(r, i) + (size_t)(r.s[i] + at)));
    };
    if (steps > 0) {
        rows_of(0, cur);
        scales_of(cur, g_first, s_even);
    }
    const W4Const kc;
    unsigned slot = 0;                         // of this step, in bytes
    const unsigned b_hop = (unsigned)p.wk * cols * 256, f_hop = (unsigned)(p.wk * p.block);
    for (int it = 0; it < iters; ++it) {
        // the residual of the thread's first output, under the products
        float res = 0.f;
        if (!GLU && p.residual && p.ks == 1) {
            const int n = row0 + (it * sets + j_set) * GR + j_row;
            if (j_set < sets && n < row1) res = residual_of(j_tok, n);
        }
        float acc[2][NB][AC];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < AC; ++c) acc[a][b][c] = 0.f;
        const int base = row0 + (it * sets + set) * GR;
        unsigned b_at[NB], b_odd[NB], f_at[NB][P == 2 ? 1 : 2];   // of the step's chunk
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int col = min(b * 8 + g, cols - 1);
            b_at[b] = smem_u32(xs) + (unsigned)(slice * cols + col) * 256 + t * 16;
            b_odd[b] = (col & 1) ? 64u : 0u;
#pragma unroll
            for (int c = 0; c < (P == 2 ? 1 : 2); ++c) {
                const int r = min(P == 2 ? b * 4 + t : b * 8 + 2 * t + c, p.block - 1);
                f_at[b][c] = (unsigned)(slice * p.block + r);
            }
        }
        auto one_step = [&](int i, const uint32_t (&use)[4], uint32_t (&fill)[4]) {
            if (i + 1 < mine) {
                scales_of(cur, g_first + (unsigned)(i + 1) * g_hop, fill);
            } else if (it + 1 < iters) {
                rows_of(it + 1, next);
                scales_of(next, g_first, fill);
            }
            cp_wait(S == 4);
            __syncwarp();
            copy_next();                       // into the slot that the step before read
            const uint32_t ta = ring_at + slot + g * 64;
            slot = (slot + WG_STEP) & (ring_bytes - 1u);
            // columns of B and tokens that there are not repeat others: what they give is not used
            float f[NB][P == 2 ? 1 : 2];       // the scales of the tokens of this lane's sums
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < (P == 2 ? 1 : 2); ++c) {
                    f[b][c] = fs[f_at[b][c]];
                    f_at[b][c] += f_hop;
                }
            // the scales of rows g and g + 8 of each tile (none behind the last group)
            const bool in = g_first + (unsigned)i * g_hop < spitch;
            const uint32_t sc[2] = {G == 128 || in ? __byte_perm(use[0], use[1], 0x5410) : 0u,
                                    G == 128 || in ? __byte_perm(use[2], use[3], 0x5410) : 0u};
            uint32_t wa[2][4], wb[2][4];       // words of rows g and g + 8 of a tile, word c for MMAs 2c and 2c + 1
            if (G == 128) {
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint4 a = lds16(ta + t * 16 + tile * 1024), b = lds16(ta + t * 16 + tile * 1024 + 512);
                    wa[tile][0] = a.x; wa[tile][1] = a.y; wa[tile][2] = a.z; wa[tile][3] = a.w;
                    wb[tile][0] = b.x; wb[tile][1] = b.y; wb[tile][2] = b.z; wb[tile][3] = b.w;
                }
            }
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                constexpr int PER = 4 / NG;    // words of a group
                if (G == 64) {
#pragma unroll
                    for (int tile = 0; tile < 2; ++tile) {
                        const uint32_t at = ta + ((2 * gi + (t >> 1)) ^ swz) * 16 + (t & 1) * 8 + tile * 1024;
                        const uint2 a = lds8(at), b = lds8(at + 512);
                        wa[tile][2 * gi] = a.x; wa[tile][2 * gi + 1] = a.y;
                        wb[tile][2 * gi] = b.x; wb[tile][2 * gi + 1] = b.y;
                    }
                }
                float d[2][NB][4];
#pragma unroll
                for (int c = gi * PER; c < (gi + 1) * PER; ++c) {
                    if (G == 32) {
#pragma unroll
                        for (int tile = 0; tile < 2; ++tile) {
                            const uint32_t at = ta + (c ^ swz) * 16 + t * 4 + tile * 1024;
                            wa[tile][c] = lds4(at);
                            wb[tile][c] = lds4(at + 512);
                        }
                    }
                    uint4 bf[NB];              // the B words of MMAs 2c and 2c + 1
#pragma unroll
                    for (int b = 0; b < NB; ++b) bf[b] = lds16(b_at[b] + (c & 1 ? -b_odd[b] : b_odd[b]) + c * 64);
                    // (a second tile without rows holds zeros: its products cost less than a branch around them)
                    uint32_t pa[2][4], pb[2][4];
#pragma unroll
                    for (int tile = 0; tile < 2; ++tile) {
                        w4_unpack(wa[tile][c], kc, pa[tile]);
                        w4_unpack(wb[tile][c], kc, pb[tile]);
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int tile = 0; tile < 2; ++tile) {
                            if (c == gi * PER) mma_first(d[tile][b], pa[tile][0], pb[tile][0], pa[tile][1], pb[tile][1], bf[b].x, bf[b].y);
                            else mma_f16(d[tile][b], pa[tile][0], pb[tile][0], pa[tile][1], pb[tile][1], bf[b].x, bf[b].y);
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int tile = 0; tile < 2; ++tile)
                            mma_f16(d[tile][b], pa[tile][2], pb[tile][2], pa[tile][3], pb[tile][3], bf[b].z, bf[b].w);
                }
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint32_t sw = NG > 1 ? __shfl_sync(0xffffffffu, sc[tile], (lane & 28) | gi) : sc[tile];
                    const float s0 = bf16_lo(sw), s1 = bf16_hi(sw);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float* e = d[tile][b];
                        float* o = acc[tile][b];
                        constexpr int L = P == 2 ? 0 : 1;
                        if (P == 2) {          // columns 2t and 2t + 1 are the two parts of one token
                            o[0] = fmaf((e[0] + e[1]) * f[b][0], s0, o[0]);
                            o[1] = fmaf((e[2] + e[3]) * f[b][0], s1, o[1]);
                        } else {
                            o[0] = fmaf(e[0] * f[b][0], s0, o[0]);
                            o[AC == 4 ? 1 : 0] = fmaf(e[1] * f[b][L], s0, o[AC == 4 ? 1 : 0]);
                            o[AC == 4 ? 2 : 0] = fmaf(e[2] * f[b][0], s1, o[AC == 4 ? 2 : 0]);
                            o[AC == 4 ? 3 : 0] = fmaf(e[3] * f[b][L], s1, o[AC == 4 ? 3 : 0]);
                        }
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) b_at[b] += b_hop;
        };
        for (int i = 0; i < mine; i += 2) {
            one_step(i, s_even, s_odd);
            if (i + 1 < mine) one_step(i + 1, s_odd, s_even);
        }
        if (mine & 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s_even[i] = s_odd[i];
        }
        if (it + 1 < iters && mine > 0) cur = next;

        // the warps' sums of the row group: [warp][token][row]
        float* rb = red + (size_t)(p.bufs > 1 ? it & 1 : 0) * WG_WARPS * MT * WG_PITCH;
        float* rw = rb + (size_t)warp * MT * WG_PITCH;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < AC; ++c) {
                    const int r = P == 2 ? b * 4 + t : b * 8 + 2 * t + (c & 1);
                    const int row = a * 16 + g + 8 * (P == 2 ? c : c >> 1);
                    rw[r * WG_PITCH + row] = acc[a][b][c];
                }
        __syncthreads();
        int r = j_tok, st2 = j_set;
        for (bool first = true; __any_sync(0xffffffffu, st2 < sets); first = false) {
            const int n = row0 + (it * sets + st2) * GR + j_row;
            const bool live = st2 < sets && n < row1;
            float v = 0.f, u = 0.f;
            if (live) {
                for (int w = tid & 3; w < p.wk; w += 4) {
                    const float* s = rb + ((size_t)(st2 * p.wk + w) * MT + r) * WG_PITCH + j_row;
                    v += s[0];
                    if (GLU) u += s[16];
                }
            }
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (GLU) {
                u += __shfl_xor_sync(0xffffffffu, u, 1);
                u += __shfl_xor_sync(0xffffffffu, u, 2);
            }
            if (live && (tid & 3) == 0) {
                if (p.ks == 1) {
                    if (!first) res = residual_of(r, n);
                    finish(r, n, v, u, res);
                } else {
                    sums[r * p.rows + n - row0] = v;
                    if (GLU) sums[(p.block + r) * p.rows + n - row0] = u;
                }
            }
            for (r += J_NEXT; r >= m; r -= m) ++st2;
        }
        // one buffer: the next row group's sums wait for this one's readers
        if (p.bufs == 1 && it + 1 < iters) __syncthreads();
    }

    if (p.ks > 1) {
        // every CTA of the cluster finishes a part of the outputs: the sums of all, in their order
        cluster_sync();
        const int nr = row1 - row0, all = nr * m;
        const int end = (int)((long long)(q + 1) * all / p.ks);
        for (int i = (int)((long long)q * all / p.ks) + tid; i < end; i += WG_THREADS) {
            const int r = i / nr, row = i - r * nr;
            const float res = residual_of(r, row0 + row);
            float v = 0.f, u = 0.f;
            for (int w = 0; w < p.ks; ++w) {
                const float* s = sums + r * p.rows + row;
                v += ld_cluster(s, w);
                if (GLU) u += ld_cluster(s + p.block * p.rows, w);
            }
            finish(r, row0 + row, v, u, res);
        }
        cluster_sync();                        // until the others have read this CTA's sums
    }
    if (!GLU && p.amax) {
        __syncthreads();
        if (tid < m) {
            if (best_s[tid]) atomicMax(p.amax + tok0 + tid, best_s[tid]);
            if (nonfinite_s[tid]) atomicOr(p.nonfinite + tok0 + tid, 1u);
        }
    }
    if (tid == 0) {
        trace_mark(tr, p.trace_id, 2);
        trace_mark(tr, p.trace_id, 3);
    }
}

// stacked matrices come from a decode step, whose activations are fp32
template <int G, int P, int NB>
const void* w4_gemv_pick(int kind) {
    if (kind == W4_ONE) return (const void*)&k_w4_gemv<G, P, NB, W4_ONE>;
    if (kind == W4_GLU) return (const void*)&k_w4_gemv<G, P, NB, W4_GLU>;
    if constexpr (P == 2) return (const void*)&k_w4_gemv<G, P, NB, W4_STACK>;
    else return nullptr;
}
template <int G>
const void* w4_gemv_kernel(int parts, int nb, int kind) {
    if (parts == 1) return nb == 1 ? w4_gemv_pick<G, 1, 1>(kind) : w4_gemv_pick<G, 1, 2>(kind);
    return nb == 1 ? w4_gemv_pick<G, 2, 1>(kind) : w4_gemv_pick<G, 2, 2>(kind);
}

}  // namespace gd
