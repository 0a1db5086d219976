// w4_gemm.cu -- the products of many tokens with 4-bit weights on the 5th-generation
// tensor cores (tcgen05.mma, sm_103a).
//
// out[t, n] = sum_k W[n, k] a[t, k].  The tensor cores take fp16, and a stored weight
// is exact in fp16: a code of 4 bits times a scale of 8 significant bits has 11, so
// once the scales of a row are brought to fp16's range by one power of two (2^11 at
// the row's largest) nothing is rounded (a scale more than 2^28 below the row's largest
// loses bits, 2^-39 of that largest).  Activations are fp16 parts, scaled by a power of two a token:
// one part for bf16 ones (8 bits fit), two for fp32.  So a bf16 call needs one MMA a
// weight tile, with fp32 sums.
//
//   k_w4_split   one CTA a token: RMSNorm's sum, the token's power of two, its parts in
//                the column order in which the words of codes come apart (w4.cuh).
//   k_w4_gemm    A = a tile of 128 output rows (TMEM lanes), B = up to 256 tokens.
//     warps 0-7  two warpgroups in turn take 64 columns of the tile: a thread has a row,
//                reads 32 bytes of codes, makes 64 fp16 weights and stores them to TMEM
//                (tcgen05.st), from where the MMA reads A: no shared memory is written,
//                and its reads are left to B
//     warp 8     codes by TMA, 128 columns a stage
//     warp 9     activations by TMA, 64 columns a stage (128-byte swizzle)
//     warp 10    tcgen05.mma kind::f16, D in TMEM (gate/up: two accumulators)
//   and warps 0-7 again for the epilogue: thread = output row, so a warp's stores of one
//   token lie side by side.
// Few tokens leave few tiles: then `ks` CTAs share the columns of a tile, leave their
// sums in the workspace, and the last to arrive adds them in order.
// Every wait is bounded; one that gives up sets FAULT_WAIT, and the CTA ends.
#include <cuda.h>
#include "w4.cuh"
#include "mma_helpers.cuh"

namespace gd {

namespace {

constexpr int WM_DQ = 8;                       // warps that make weights, and write results
constexpr int WM_THREADS = (WM_DQ + 3) * 32;
constexpr int WM_CODES = 128 * 64;             // bytes of a codes stage: 128 rows x 128 columns
constexpr int WM_MAX_SC = 16, WM_MAX_SB = 12;
constexpr int WM_SMEM = 200 * 1024;            // for both rings
constexpr int WM_MAX_NT = 256;

struct WmParams {
    CUtensorMap codes[2];      // [n, k / 2] bytes, box [64, 128], 64-byte swizzle
    CUtensorMap x;             // [parts * tokens, kp] fp16, box [64, nt], 128-byte swizzle
    const __nv_bfloat16* scales[2];
    const float* factor;       // [tokens]
    const void* residual;
    void* out;
    long long residual_stride, out_stride;
    int N, K, tokens, nt, ks, ksteps, sc, sb, na, act, out_f32;
    bool wide;                 // scales can be read eight at a time
    float* part;
    unsigned* count;
    unsigned* err;
};

__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// D (+)= A B over 64 columns by the warp's elected lane: A in TMEM (8 columns a step of 16), B K-major in shared memory
// (128-byte swizzle, 32 bytes a step).  acc 0: D starts anew
constexpr uint32_t WM_DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ void mma_64(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred e, p, t;\n .reg .b64 y;\n .reg .b32 a;\n setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
                 " mov.b32 a, %1;\n mov.b64 y, {%2, %3};\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, p;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n}\n" ::"r"(d), "r"(a),
                 "r"(((b & 0x3FFFFu) >> 4) | 1u << 16), "r"(WM_DESC_HI), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
                 : "memory");
}

// a row's scales are multiplied by 2^(11 - e), 2^e the power of two at or below the largest of them: weights below 2^15
__device__ __forceinline__ float row_up(int e) { return __uint_as_float((uint32_t)(265 - e) << 23); }
__device__ __forceinline__ float row_down(int e) { return __uint_as_float((uint32_t)(e - 11) << 23); }
// a scale's bf16 bits as the scaled fp16 in both halves
__device__ __forceinline__ uint32_t scale_pair(uint32_t bits, float up) {
    const float s = __uint_as_float(bits << 16) * up;
    return w4_pack_half(s, s);
}
__device__ __forceinline__ uint32_t pick16(const uint4& w, int i) {   // element i (0 .. 7) of eight
    const uint32_t lo = i & 2 ? w.y : w.x, hi = i & 2 ? w.w : w.z, v = i & 4 ? hi : lo;
    return i & 1 ? v >> 16 : v & 0xffffu;
}

// G: columns of a group; P: fp16 parts of an activation
template <int G, int P, bool GLU>
__global__ void __launch_bounds__(WM_THREADS, 1) k_w4_gemm(const __grid_constant__ WmParams p) {
    constexpr int MATS = GLU ? 2 : 1;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t codes_full[WM_MAX_SC], codes_empty[WM_MAX_SC], x_full[WM_MAX_SB], x_empty[WM_MAX_SB];
    __shared__ __align__(8) uint64_t a_full[8], a_empty[8], done;
    __shared__ uint32_t tmem;
    __shared__ int aborted, last_s;
    __shared__ int row_e[MATS][128];
    __shared__ float tok_f[WM_MAX_NT];
    volatile int* ab = &aborted;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x, blk = blockIdx.y, split = blockIdx.z;
    const int row0 = tile * 128, tok0 = blk * p.nt, m = min(p.nt, p.tokens - tok0);
    // this split's steps of 64 columns, an even number but for the last split's
    const int pairs = (p.ksteps + 1) >> 1;
    const int s0 = 2 * (int)((long long)split * pairs / p.ks);
    const int s1 = min(p.ksteps, 2 * (int)((long long)(split + 1) * pairs / p.ks));
    const int n = s1 - s0;
    const int xbytes = p.nt * P * 128, cbytes = WM_CODES * MATS;
    unsigned char* codes_s = smem;
    unsigned char* x_s = smem + (size_t)p.sc * cbytes;
    const int spitch = p.K / G;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int s = 0; s < p.sc; ++s) {
            mbar_init(&codes_full[s], 1);
            mbar_init(&codes_empty[s], WM_DQ);
        }
        for (int s = 0; s < p.sb; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 1);
        }
        for (int s = 0; s < p.na; ++s) {
            mbar_init(&a_full[s], WM_DQ / 2);
            mbar_init(&a_empty[s], 1);
        }
        mbar_init(&done, 1);
        aborted = 0;
        mbar_fence_init();
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t dt = tmem, at0 = dt + (uint32_t)(p.nt * MATS);   // accumulators, then the ring of A
    auto give_up = [&]() {
        *ab = 1;
        atomicOr(p.err, FAULT_WAIT);
    };

    if (warp == WM_DQ) {
        // ---- codes ----
        int issued = 0;
        const int stages = (n + 1) >> 1;
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                const int slot = s % p.sc;
                if (*ab) break;
                if (s >= p.sc && !mbar_wait(&codes_empty[slot], (uint32_t)(s / p.sc - 1) & 1u)) {
                    give_up();
                    break;
                }
                mbar_arrive_expect_tx(&codes_full[slot], (uint32_t)cbytes);
#pragma unroll
                for (int i = 0; i < MATS; ++i)
                    tma_load_2d(codes_s + (size_t)slot * cbytes + i * WM_CODES, &p.codes[i], (s0 + 2 * s) * 32, row0, &codes_full[slot]);
                issued = s + 1;
            }
            // no copy may still be landing when the CTA exits
            for (int s = max(0, issued - p.sc); s < issued; ++s)
                if (!mbar_wait(&codes_full[s % p.sc], (uint32_t)(s / p.sc) & 1u)) give_up();
        }
        __syncwarp();
    } else if (warp == WM_DQ + 1) {
        // ---- activations ----
        int issued = 0;
        if (lane == 0) {
            pdl_wait();   // k_w4_split has written them
            for (int s = 0; s < n; ++s) {
                const int slot = s % p.sb;
                if (*ab) break;
                if (s >= p.sb && !mbar_wait(&x_empty[slot], (uint32_t)(s / p.sb - 1) & 1u)) {
                    give_up();
                    break;
                }
                mbar_arrive_expect_tx(&x_full[slot], (uint32_t)xbytes);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    tma_load_2d(x_s + (size_t)slot * xbytes + i * p.nt * 128, &p.x, (s0 + s) * 64, i * p.tokens + tok0, &x_full[slot]);
                issued = s + 1;
            }
            for (int s = max(0, issued - p.sb); s < issued; ++s)
                if (!mbar_wait(&x_full[s % p.sb], (uint32_t)(s / p.sb) & 1u)) give_up();
        }
        __syncwarp();
    } else if (warp == WM_DQ + 2) {
        // ---- products ----
        const uint32_t idesc = (1u << 4) | ((uint32_t)(p.nt >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        for (int s = 0; s < n; ++s) {
            const int sa = s % p.na, sx = s % p.sb;
            const bool ok = !*ab && mbar_wait(&a_full[sa], (uint32_t)(s / p.na) & 1u) && mbar_wait(&x_full[sx], (uint32_t)(s / p.sb) & 1u);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            fence_after();
            const uint32_t xb = smem_u32(x_s + (size_t)sx * xbytes);
#pragma unroll
            for (int i = 0; i < MATS; ++i)
#pragma unroll
                for (int q = 0; q < P; ++q)
                    mma_64(dt + (uint32_t)(i * p.nt), at0 + (uint32_t)((sa * MATS + i) * 32), xb + (uint32_t)(q * p.nt * 128), idesc,
                           s > 0 || q > 0 ? 1u : 0u);
            commit(&a_empty[sa]);
            commit(&x_empty[sx]);
        }
        commit(&done);
    } else {
        // ---- weights ----
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;   // TMEM lane = tile row
        // the rows' powers of two: a warp takes 16 rows of each matrix, its lanes the scales of a row
        const int g0 = s0 * 64 / G, g1 = min(spitch, (s1 * 64 + G - 1) / G);
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
#pragma unroll 4
            for (int j = 0; j < 16; ++j) {
                const int rr = warp * 16 + j;
                uint32_t top = 0;
                if (row0 + rr < p.N) {
                    const unsigned short* s = reinterpret_cast<const unsigned short*>(p.scales[i]) + (size_t)(row0 + rr) * spitch;
                    for (int c = g0 + lane; c < g1; c += 32) {
                        const uint32_t b = __ldg(s + c) & 0x7fffu;
                        top = max(top, b < 0x7f80u ? b : 0u);
                    }
                }
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) row_e[i][rr] = min(max((int)(top >> 7), 12), 254);
            }
        }
        named_sync(1, WM_DQ * 32);
        const bool in = row0 + r < p.N;
        float up[MATS];
        const unsigned short* sp[MATS];
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
            up[i] = row_up(row_e[i][r]);
            sp[i] = reinterpret_cast<const unsigned short*>(p.scales[i]) + (size_t)(in ? row0 + r : 0) * spitch;
        }
        // eight scales of the row at a time, the next eight under way
        constexpr int WIN = 8 * G / 64;   // steps of eight groups
        uint4 sw[MATS], sn[MATS];
        int win = -1;
        auto load_win = [&](int i, int w) {
            return w * 8 < spitch ? __ldg(reinterpret_cast<const uint4*>(sp[i]) + w) : make_uint4(0u, 0u, 0u, 0u);
        };
        const int swz = (r >> 1) & 3;
        for (int s = wg; s < n; s += 2) {
            const int cs = s >> 1, slot = cs % p.sc, sa = s % p.na, step = s0 + s;
            uint32_t sc[MATS][G == 32 ? 2 : 1];
            if (p.wide) {
                const int w = step / WIN;
                if (w != win) {
#pragma unroll
                    for (int i = 0; i < MATS; ++i) {
                        sw[i] = win < 0 ? load_win(i, w) : sn[i];
                        sn[i] = load_win(i, w + 1);
                    }
                    win = w;
                }
#pragma unroll
                for (int i = 0; i < MATS; ++i)
#pragma unroll
                    for (int h = 0; h < (G == 32 ? 2 : 1); ++h)
                        sc[i][h] = scale_pair(pick16(sw[i], (G == 32 ? step * 2 + h : step * 64 / G) & 7), up[i]);
            } else {
#pragma unroll
                for (int i = 0; i < MATS; ++i)
#pragma unroll
                    for (int h = 0; h < (G == 32 ? 2 : 1); ++h) {
                        const int c = G == 32 ? step * 2 + h : step * 64 / G;
                        sc[i][h] = c < spitch ? scale_pair(__ldg(sp[i] + c), up[i]) : 0u;
                    }
            }
            bool ok = !*ab && mbar_wait(&codes_full[slot], (uint32_t)(cs / p.sc) & 1u);
            uint4 q[MATS][2];
#pragma unroll
            for (int i = 0; i < MATS; ++i) {
                const unsigned char* row = codes_s + (size_t)slot * cbytes + i * WM_CODES + r * 64;
                q[i][0] = *reinterpret_cast<const uint4*>(row + (((2 * wg) ^ swz) << 4));
                q[i][1] = *reinterpret_cast<const uint4*>(row + (((2 * wg + 1) ^ swz) << 4));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&codes_empty[slot]);
            if (s >= p.na) ok = ok && mbar_wait(&a_empty[sa], (uint32_t)(s / p.na - 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            fence_after();
#pragma unroll
            for (int i = 0; i < MATS; ++i) {
                uint32_t a[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w[4] = {q[i][h].x, q[i][h].y, q[i][h].z, q[i][h].w};
                    const uint32_t f = sc[i][G == 32 ? h : 0];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pr[4];
                        w4_unpack(w[c], pr);
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[h * 16 + c * 4 + e] = w4_hmul(pr[e], f);
                    }
                }
                tm_st32(at0 + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)((sa * MATS + i) * 32), a);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[sa]);
        }
        // an odd number of steps: the second warpgroup leaves its half of the last stage unread
        if ((n & 1) && wg == 1 && lane == 0) mbar_arrive(&codes_empty[((n - 1) >> 1) % p.sc]);

        // ---- epilogue ----
        pdl_wait();
        for (int i = tid; i < m; i += WM_DQ * 32) tok_f[i] = __ldcg(p.factor + tok0 + i);
        named_sync(1, WM_DQ * 32);
        const bool okd = mbar_wait(&done, 0u);
        if (!okd) give_up();
        fence_after();
        const bool live = okd && !*ab;
        const int nn = row0 + r;
        float down[MATS];
#pragma unroll
        for (int i = 0; i < MATS; ++i) down[i] = row_down(row_e[i][r]);
        auto put = [&](int t, float v, float u) {   // token t of the block; sums in true size
            if (GLU) v = w4_glu(p.act, v, u);
            else if (p.residual) v += w4_load1(p.residual, p.out_f32, (size_t)(tok0 + t) * p.residual_stride + nn);
            w4_store1(p.out, p.out_f32, (size_t)(tok0 + t) * p.out_stride + nn, v);
        };
        // the smaller factor first: no step leaves fp32's range unless the result does
        auto sized = [&](float v, float a, float b) { return v * fminf(a, b) * fmaxf(a, b); };
        if (__all_sync(0xffffffffu, live)) {
            for (int c = wg * 16; c < p.nt; c += 32) {
                if (c >= m) break;
                uint32_t d[MATS][16];
#pragma unroll
                for (int i = 0; i < MATS; ++i) tm_ld16(dt + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(i * p.nt + c), d[i]);
                float res[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    res[e] = !GLU && p.ks == 1 && p.residual && in && c + e < m
                                 ? w4_load1(p.residual, p.out_f32, (size_t)(tok0 + c + e) * p.residual_stride + nn) : 0.f;
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int e = 0; e < 16; ++e) {
#pragma unroll
                    for (int i = 0; i < MATS; ++i) asm volatile("" : "+r"(d[i][e]));
                    if (!in || c + e >= m) continue;
                    const float f = tok_f[c + e];
                    const float v = sized(__uint_as_float(d[0][e]), down[0], f);
                    const float u = GLU ? sized(__uint_as_float(d[MATS - 1][e]), down[MATS - 1], f) : 0.f;
                    if (p.ks > 1) {
                        float* o = p.part + ((size_t)split * p.tokens + tok0 + c + e) * p.N * MATS + nn;
                        o[0] = v;
                        if (GLU) o[p.N] = u;
                    } else {
                        w4_store1(p.out, p.out_f32, (size_t)(tok0 + c + e) * p.out_stride + nn, GLU ? w4_glu(p.act, v, u) : v + res[e]);
                    }
                }
            }
        }
        if (p.ks > 1) {
            __threadfence();
            named_sync(1, WM_DQ * 32);
            if (tid == 0) {
                unsigned* cnt = p.count + (size_t)blk * gridDim.x + tile;
                const unsigned before = atomicAdd(cnt, 1u);
                last_s = before == (unsigned)p.ks - 1u;
                if (last_s) *cnt = 0u;         // ready for the next call
            }
            named_sync(1, WM_DQ * 32);
            if (last_s) {
                __threadfence();
                if (in) {
                    for (int t = wg; t < m; t += 2) {
                        float v = 0.f, u = 0.f;
                        for (int w = 0; w < p.ks; ++w) {
                            const float* o = p.part + ((size_t)w * p.tokens + tok0 + t) * p.N * MATS + nn;
                            v += __ldcg(o);
                            if (GLU) u += __ldcg(o + p.N);
                        }
                        put(t, v, u);
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(dt) : "memory");
    }
}

// ---- the activations' parts ----
constexpr int WS_THREADS = 256;

template <int P>
__global__ void __launch_bounds__(WS_THREADS) k_w4_split(const void* x, long long stride, bool x_f32, const void* gain, bool gain_f32,
                                                         float eps, int K, int kp, int tokens, __half* parts, float* factor) {
    __shared__ float ss_s[WS_THREADS / 32];
    __shared__ uint32_t top_s[WS_THREADS / 32];
    pdl_trigger();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto load = [&](int c, float (&v)[8], float* ss) {
        const float4 a = w4_load4(x, x_f32, (size_t)t * stride + c), b = w4_load4(x, x_f32, (size_t)t * stride + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        if (gain) {
            if (ss) {
#pragma unroll
                for (int e = 0; e < 8; ++e) *ss = fmaf(v[e], v[e], *ss);
            }
            const float4 g = w4_load4(gain, gain_f32, c), h = w4_load4(gain, gain_f32, c + 4);
            v[0] *= g.x; v[1] *= g.y; v[2] *= g.z; v[3] *= g.w; v[4] *= h.x; v[5] *= h.y; v[6] *= h.z; v[7] *= h.w;
        }
    };
    float ss = 0.f;
    uint32_t top = 0;
    for (int c = tid * 8; c < K; c += WS_THREADS * 8) {
        float v[8];
        load(c, v, &ss);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, w4_finite_bits(v[e]));
    }
    ss = warp_sum(ss);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
        ss_s[warp] = ss;
        top_s[warp] = top;
    }
    __syncthreads();
    ss = 0.f;
    top = 0;
#pragma unroll
    for (int w = 0; w < WS_THREADS / 32; ++w) {
        ss += ss_s[w];
        top = max(top, top_s[w]);
    }
    const int e = w4_exponent(top);
    const float up = w4_up(e);
    if (tid == 0) factor[t] = w4_down(e) * (gain ? 1.0f / sqrtf(ss / (float)K + eps) : 1.0f);
    for (int c = tid * 8; c < kp; c += WS_THREADS * 8) {
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (c < K) {
            float v[8];
            load(c, v, nullptr);
            uint32_t* h = &hi.x;
            uint32_t* l = &lo.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = v[j] * up, b = v[j + 4] * up;
                h[j] = w4_pack_half(a, b);
                if (P == 2) l[j] = w4_rest(a, b, h[j]);
            }
        }
        *reinterpret_cast<uint4*>(parts + (size_t)t * kp + c) = hi;
        if (P == 2) *reinterpret_cast<uint4*>(parts + ((size_t)tokens + t) * kp + c) = lo;
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn.store(f = reinterpret_cast<EncodeFn>(ptr), std::memory_order_release);
    }
    return f;
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long rows, long long cols, long long pitch, int box_cols,
            int box_rows, CUtensorMapSwizzle swz) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, estr[2] = {1u, 1u};
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G>
const void* gemm_kernel(int P, bool glu) {
    if (P == 1) return glu ? (const void*)&k_w4_gemm<G, 1, true> : (const void*)&k_w4_gemm<G, 1, false>;
    return glu ? (const void*)&k_w4_gemm<G, 2, true> : (const void*)&k_w4_gemm<G, 2, false>;
}

const void* kernel_of(const W4Gemm& g) {
    const int P = g.c.x_f32 ? 2 : 1;
    switch (g.c.group()) {
        case 32: return gemm_kernel<32>(P, g.c.glu);
        case 64: return gemm_kernel<64>(P, g.c.glu);
        default: return gemm_kernel<128>(P, g.c.glu);
    }
}

int round_up(int v, int to) { return (v + to - 1) / to * to; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

cudaError_t w4_gemm_plan(W4Gemm* g, int num_sms) {
    const W4Call& c = g->c;
    const int P = c.x_f32 ? 2 : 1, mats = c.glu ? 2 : 1;
    const int tiles = (c.n() + 127) / 128, ksteps = (c.k() + 63) / 64, most = P * mats > 1 ? 128 : 256;
    // Tokens of a tile and CTAs along k: the least time of the longest CTA, in clocks.  A step of 64 columns takes the
    // tensor cores 2 clocks a token, part and matrix, its weights 150 a matrix to make; a CTA starts and ends in about
    // 4000, and a split adds the writing and reading of its sums
    double best = -1.0;
    const int least = (c.tokens + most - 1) / most;
    for (int blocks = least; blocks <= least + 8; ++blocks) {
        const int nt = round_up((c.tokens + blocks - 1) / blocks, 16), used = (c.tokens + nt - 1) / nt;
        for (int ks = 1; ks <= 16; ++ks) {
            if (ks > 1 && (ksteps / ks < 8 || (long long)tiles * used > DEC_W4_COUNTER_BYTES / 4)) break;
            const double waves = (double)(((long long)tiles * used * ks + num_sms - 1) / num_sms);
            const double step = 2.0 * nt * P * mats > 150.0 * mats ? 2.0 * nt * P * mats : 150.0 * mats;
            const double t = waves * ((double)((ksteps + ks - 1) / ks) * step + 4000.0 + 12.0 * nt * mats) +
                             (ks > 1 ? 2500.0 + 10.0 * nt * mats * ks : 0.0);
            if (best < 0.0 || t < best) {
                best = t;
                g->nt = nt;
                g->ks = ks;
            }
        }
        if (nt <= 16) break;
    }
    g->kp = round_up(c.k(), 64);
    g->ksteps = ksteps;
    const void* fn = kernel_of(*g);
    static OncePerDevice once[3][2][2];
    return once[c.group() == 32 ? 0 : c.group() == 64 ? 1 : 2][P - 1][c.glu].run([&] { return raise_smem_cap(fn); });
}

size_t w4_gemm_bytes(const W4Gemm& g) {
    const W4Call& c = g.c;
    const int P = c.x_f32 ? 2 : 1;
    return round256((size_t)P * c.tokens * g.kp * 2) + round256((size_t)c.tokens * 4) +
           (g.ks > 1 ? (size_t)g.ks * c.tokens * c.n() * (c.glu ? 2 : 1) * 4 : 0);
}

cudaError_t w4_gemm_launch(const W4Gemm& g, cudaStream_t s) {
    const W4Call& c = g.c;
    const int P = c.x_f32 ? 2 : 1, mats = c.glu ? 2 : 1;
    __half* parts = (__half*)g.ws;
    float* factor = (float*)((char*)g.ws + round256((size_t)P * c.tokens * g.kp * 2));
    WmParams p{};
    for (int i = 0; i < 2; ++i) {
        const W4Matrix& w = c.w[i < mats ? i : 0];
        if (!encode(&p.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.n, w.k / 2, w.k / 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
        p.scales[i] = (const __nv_bfloat16*)w.scales;
    }
    if (!encode(&p.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, parts, (long long)P * c.tokens, g.kp, 2ll * g.kp, 64, g.nt,
                CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    p.factor = factor;
    p.residual = c.residual;
    p.out = c.out;
    p.residual_stride = c.residual_stride;
    p.out_stride = c.out_stride;
    p.N = c.n();
    p.K = c.k();
    p.tokens = c.tokens;
    p.nt = g.nt;
    p.ks = g.ks;
    p.ksteps = g.ksteps;
    p.act = c.act;
    p.out_f32 = c.out_f32;
    p.wide = (c.k() / c.group()) % 8 == 0 && ((uintptr_t)p.scales[0] & 15) == 0 && ((uintptr_t)p.scales[1] & 15) == 0;
    p.part = (float*)((char*)factor + round256((size_t)c.tokens * 4));
    p.count = g.count;
    p.err = c.err;
    // the rings: activations first, the rest for codes
    const int xb = g.nt * P * 128, cb = WM_CODES * mats;
    p.sb = (WM_SMEM - 4 * cb) / xb;
    if (p.sb > WM_MAX_SB) p.sb = WM_MAX_SB;
    p.sc = (WM_SMEM - p.sb * xb) / cb;
    if (p.sc > WM_MAX_SC) p.sc = WM_MAX_SC;
    p.na = (512 - g.nt * mats) / (32 * mats);
    if (p.na > 8) p.na = 8;
    if (p.sb < 2 || p.sc < 2 || p.na < 2) return cudaErrorInvalidValue;

    if (P == 1)
        k_w4_split<1><<<c.tokens, WS_THREADS, 0, s>>>(c.x, c.x_stride, c.x_f32, c.gain, c.gain_f32, c.eps, c.k(), g.kp, c.tokens, parts, factor);
    else
        k_w4_split<2><<<c.tokens, WS_THREADS, 0, s>>>(c.x, c.x_stride, c.x_f32, c.gain, c.gain_f32, c.eps, c.k(), g.kp, c.tokens, parts, factor);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((c.n() + 127) / 128, (c.tokens + g.nt - 1) / g.nt, g.ks);
    cfg.blockDim = dim3(WM_THREADS);
    cfg.dynamicSmemBytes = (size_t)p.sb * xb + (size_t)p.sc * cb + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];   // starts while k_w4_split runs: codes and scales do not depend on it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, kernel_of(g), args);
}

}  // namespace gd
