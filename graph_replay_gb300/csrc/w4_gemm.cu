// w4_gemm.cu -- the products of many tokens with 4-bit weights on the 5th-generation
// tensor cores (tcgen05.mma, sm_103a).
//
// out[t, n] = sum_k W[n, k] a[t, k].  The tensor cores take fp16, and a stored weight
// is exact in fp16: a code of 4 bits times a scale of 8 significant bits has 11, so
// once the scales of a row are brought to fp16's range by one power of two (2^10 at
// the row's largest) nothing is rounded (a scale more than 2^27 below the row's largest
// loses bits, 2^-38 of that largest).  Activations are fp16 parts, scaled by a power of
// two a token: one part for bf16 ones (8 bits fit), two for fp32 ones and for normed ones
// (the product with a gain has up to 24 bits whatever the types), and for fp32 results.
//
//   k_w4_split   one CTA a token: RMSNorm's sum, the token's power of two, its parts in
//                the column order in which the words of codes come apart (w4.cuh).
//   k_w4_gemm    A = two tiles (WIDE: one) of 128 output rows (TMEM lanes): 256 rows of one matrix, or
//                128 rows each of gate and up; B = up to 128 tokens, read from shared memory
//                once for both.  A step is 128 columns:
//     warps 0-15 a warpgroup takes one tile and one half of the step's columns: a thread has
//                a row, reads 32 bytes of codes, makes 64 fp16 weights and stores them to
//                TMEM (tcgen05.st), from where the MMA reads A: no shared memory is written,
//                and its reads are left to B
//     warp 16    codes by TMA (64-byte swizzle)
//     warp 17    activations by TMA (128-byte swizzle)
//     warps 18-19 tcgen05.mma kind::f16, a tile each, accumulators in TMEM
//   and warps 0-15 again for the epilogue: thread = output row, so a warp's stores of one
//   token lie side by side.
// Two parts are twice as many columns of one MMA (an MMA of 64
// columns takes as long as one of 128 when A lies in TMEM).  The tensor core cuts its fp32
// sums off instead of rounding them, so these accumulators are folded into registers every
// WM_FOLD steps, with rounding; the two tiles' turns lie half of that apart, and one tile's
// MMAs run while the other's sums are taken.
// Few tokens leave few tiles: then a cluster of `ks` CTAs shares the columns of a tile,
// and each of them adds the sums of a part of the tokens from the others' shared memory,
// in order.
// Every wait is bounded; one that gives up sets FAULT_WAIT, and the CTA ends.
//
// Measured, in captures: 4095 bf16 tokens, 14336 -> 4096: 437 us, 1100 TFLOP/s (a library
// product of 16-bit weights: 1918).  1000 fp32 tokens, gate and up 14336 x 4096: 513 us, 458
// TFLOP/s of result, twice that in the tensor cores.  64 bf16 tokens, 4096 x 4096: 21.3 us; 40
// with a norm (two parts), 6144 x 4096: 26.9 us, 96 CTAs of clusters of four.
// A step takes about 1700 clocks, the MMAs of 128 tokens 1024 of them; making the weights takes
// 1300 (720 of them arithmetic, four warps a scheduler, and 100 to 250 for each wait even when
// there is nothing to wait for).  The tensor pipe is active 42 % of a launch of 1024 tokens.
// Many tokens of two parts (WIDE): one row tile and two blocks of tokens a CTA, 64 gate and 64 up rows;
// two of the warpgroups make a step's weights, the other two the next step's.
#include <cuda.h>
#include "w4.cuh"
#include "mma_helpers.cuh"

namespace gd {

namespace {

constexpr int WM_DQ = 16;                      // warps that make weights, and write results: four warpgroups
constexpr int WM_THREADS = (WM_DQ + 4) * 32;
constexpr int WM_MAX_SC = 12, WM_MAX_SX = 12, WM_MAX_SA = 4;
constexpr int WM_SMEM = 200 * 1024;            // for both rings
constexpr int WM_ROWS = 257;                   // of a split's sums of one token: 256, and one against bank conflicts
// two parts: steps of an accumulator. 2: errors as of a plain fp32 product, 4: up to 4 times that; 1 % slower than 4
constexpr int WM_FOLD = 2;
// one part: columns of an accumulator at most
constexpr int WM_UNFOLDED = 32768;

// two parts: stages of 64 columns, and half as many tokens
constexpr int wm_tokens(int P) { return P == 2 ? 64 : 128; }
// wide (two parts): one row tile and two blocks of tokens
constexpr int wm_codes(bool wide) { return (wide ? 1 : 2) * 128 * 64; }   // bytes of a codes stage: 128 rows x 128 columns a tile
constexpr int wm_stage(bool wide, int nt) { return nt * (wide ? 512 : 256); }   // bytes: 128 columns of one part or 64 of two
constexpr int wm_rows(bool glu, bool wide) { return (glu ? 128 : 256) >> (wide ? 1 : 0); }   // output rows of a CTA

struct WmParams {
    CUtensorMap codes[2];      // [n, k / 2] bytes, box [64, 128] (WIDE and GLU: [64, 64]), 64-byte swizzle
    CUtensorMap x;             // [parts * tokens, kp] fp16, box [64, nt], 128-byte swizzle
    const __nv_bfloat16* scales[2];
    const float* factor;       // [tokens]
    const void* residual;
    void* out;
    long long residual_stride, out_stride;
    int N, K, tokens, nt, ks, steps, sc, sx, sa, act, out_f32;
    bool wide;                 // scales can be read eight at a time
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
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
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
// D (+)= A B over 64 columns: A in TMEM (8 columns a step of 16), B K-major in shared memory (128-byte swizzle, 32 bytes a
// step; `b` is the low word of its descriptor).  acc 0: D starts anew.  The whole warp comes here with the same operands and
// its elected lane issues: 100 clocks for four MMAs, 300 from the code of a single lane
constexpr uint32_t WM_DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t wm_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ void mma_64(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred e, p, t;\n .reg .b64 y;\n .reg .b32 a;\n setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
                 " mov.b32 a, %1;\n mov.b64 y, {%2, %3};\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, p;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(WM_DESC_HI),
                 "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
                 : "memory");
}

// where a ring stands: a division by its length would take longer than a step
struct Ring {
    int slot = 0;
    uint32_t odd = 0;          // parity of the rounds gone through
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) {
            slot = 0;
            odd ^= 1u;
        }
    }
};

// a row's scales are multiplied by 2^(10 - e), 2^e the power of two at or below the largest of them: weights below 2^14
__device__ __forceinline__ float row_up(int e) { return __uint_as_float((uint32_t)(264 - e) << 23); }
__device__ __forceinline__ float row_down(int e) { return __uint_as_float((uint32_t)(e - 10) << 23); }
// a scale's bf16 bits as the scaled fp16 in both halves
__device__ __forceinline__ uint32_t scale_pair(uint32_t bits, float up) {
    const float s = __uint_as_float(bits << 16) * up;
    return w4_pack_half(s, s);
}
// The columns (j, j + 4) of a word times a scale s, f = (s, s) and f24 = (-24 s, -24 s), exact.  Two pairs as in w4_unpack,
// then times s; the other two with the code moved to the top of the mantissa of 16, where (16 + (q + 8)) s - 24 s is one
// fused step (24 s has 10 significant bits): so the half-precision and the integer pipe get as much each
__device__ __forceinline__ void unpack_scaled(uint32_t w, const W4Const& k, uint32_t sixteen, uint32_t f, uint32_t f24, uint32_t* o) {
    o[0] = w4_hmul(w4_hsub(w4_and_xor<0x000f000fu>(w, k.low), k.low), f);
    o[1] = w4_hmul(w4_hfma(w4_and_xor<0x00f000f0u>(w, k.high), k.part, k.less), f);
    o[2] = w4_hfma(w4_and_xor<0x03c003c0u>(w >> 2, sixteen), f, f24);
    o[3] = w4_hfma(w4_and_xor<0x03c003c0u>(w >> 6, sixteen), f, f24);
}
__device__ __forceinline__ uint32_t pick16(const uint4& w, int i) {   // element i (0 .. 7) of eight
    const uint32_t lo = i & 2 ? w.y : w.x, hi = i & 2 ? w.w : w.z, v = i & 4 ? hi : lo;
    return i & 1 ? v >> 16 : v & 0xffffu;
}

// G: columns of a group; P: fp16 parts of an activation; WIDE: one row tile and two blocks of tokens
template <int G, int P, bool GLU, bool WIDE>
__global__ void __launch_bounds__(WM_THREADS, 1) k_w4_gemm(const __grid_constant__ WmParams p) {
    constexpr int ROWS = wm_rows(GLU, WIDE), CODES = wm_codes(WIDE);
    static_assert(P == 2 || !WIDE, "");
    constexpr int XH = P;                      // activation stages of a step
    constexpr int MAKERS = WIDE ? WM_DQ / 2 : WM_DQ;   // warps that make a step's weights
    constexpr int EACH = WIDE ? 2 : 1;         // a warpgroup's steps lie so far apart
    constexpr int AC = WIDE ? 64 : 128;        // TMEM columns of a step's weights
    constexpr int APART = WM_FOLD / 2;         // steps between the two accumulators' turns (WIDE: as the makers' steps)
    constexpr bool FOLD = P == 2;
    constexpr int NS = G == 32 ? 2 : 1;        // scales of a thread's 64 columns
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t codes_full[WM_MAX_SC], codes_empty[WM_MAX_SC], x_full[WM_MAX_SX], x_empty[WM_MAX_SX];
    __shared__ __align__(8) uint64_t a_full[WM_MAX_SA], a_empty[WM_MAX_SA], d_full[2], d_empty[2], done[2];
    __shared__ uint32_t tmem;
    __shared__ int aborted;
    __shared__ int row_e[WIDE ? 1 : 2][128];
    __shared__ float tok_f[WIDE ? 256 : 128];
    volatile int* ab = &aborted;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x % p.ks, tile = blockIdx.x / p.ks, blk = blockIdx.y;
    const int row0 = tile * ROWS, nblk = WIDE ? 2 * p.nt : p.nt, tok0 = blk * nblk, m = min(nblk, p.tokens - tok0);
    const int s0 = (int)((long long)split * p.steps / p.ks), s1 = (int)((long long)(split + 1) * p.steps / p.ks);
    const int n = s1 - s0;                     // steps of this split, >= 1
    const int xbytes = wm_stage(WIDE, p.nt);
    unsigned char* codes_s = smem;
    unsigned char* x_s = smem + (size_t)p.sc * CODES;
    const int spitch = p.K / G;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int s = 0; s < p.sc; ++s) {
            mbar_init(&codes_full[s], 1);
            mbar_init(&codes_empty[s], MAKERS);
        }
        for (int s = 0; s < p.sx; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 2);         // both issuing warps
        }
        for (int s = 0; s < p.sa; ++s) {
            mbar_init(&a_full[s], MAKERS);
            mbar_init(&a_empty[s], 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&d_full[s], 1);          // of a tile, or (WIDE) of a block of tokens
            mbar_init(&d_empty[s], WM_DQ / 2);
            mbar_init(&done[s], 1);
        }
        aborted = 0;
        mbar_fence_init();
    }
    fence_before();
    __syncthreads();
    fence_after();
    // TMEM columns: accumulators (of a tile: its tokens' sums, of the second parts behind those of the first), then the
    // ring of A
    const int dcols = p.nt * P;
    const uint32_t dt = tmem, at0 = dt + (uint32_t)(2 * dcols);
    auto give_up = [&]() {
        *ab = 1;
        atomicOr(p.err, FAULT_WAIT);
    };

    if (warp == WM_DQ) {
        // ---- codes ----
        if (lane == 0) {
            Ring r;
            int issued = 0;
            for (int s = 0; s < n; ++s, r.next(p.sc)) {
                if (*ab) break;
                if (s >= p.sc && !mbar_wait(&codes_empty[r.slot], r.odd ^ 1u)) {
                    give_up();
                    break;
                }
                unsigned char* dst = codes_s + (size_t)r.slot * CODES;
                mbar_arrive_expect_tx(&codes_full[r.slot], CODES);
                tma_load_2d(dst, &p.codes[0], (s0 + s) * 64, row0, &codes_full[r.slot]);
                if (GLU || !WIDE)
                    tma_load_2d(dst + CODES / 2, &p.codes[1], (s0 + s) * 64, GLU ? row0 : row0 + 128, &codes_full[r.slot]);
                issued = s + 1;
            }
            // no copy may still be landing when the CTA exits
            for (int s = max(0, issued - p.sc); s < issued; ++s)
                if (!mbar_wait(&codes_full[s % p.sc], (uint32_t)(s / p.sc) & 1u)) give_up();
        }
        __syncwarp();
    } else if (warp == WM_DQ + 1) {
        // ---- activations: a step is one stage of 128 columns, or two of 64 with both parts ----
        if (lane == 0) {
            pdl_wait();   // k_w4_split has written them
            Ring r;
            int issued = 0;
            for (int s = 0; s < n * XH; ++s, r.next(p.sx)) {
                if (*ab) break;
                if (s >= p.sx && !mbar_wait(&x_empty[r.slot], r.odd ^ 1u)) {
                    give_up();
                    break;
                }
                unsigned char* dst = x_s + (size_t)r.slot * xbytes;
                mbar_arrive_expect_tx(&x_full[r.slot], (uint32_t)xbytes);
#pragma unroll
                for (int i = 0; i < (WIDE ? 4 : 2); ++i)   // WIDE: of each block of tokens both parts
                    tma_load_2d(dst + i * p.nt * 128, &p.x, P == 2 ? (s0 * 2 + s) * 64 : (s0 + s) * 128 + i * 64,
                                P == 2 ? (i & 1) * p.tokens + tok0 + (i >> 1) * p.nt : tok0, &x_full[r.slot]);
                issued = s + 1;
            }
            for (int s = max(0, issued - p.sx); s < issued; ++s)
                if (!mbar_wait(&x_full[s % p.sx], (uint32_t)(s / p.sx) & 1u)) give_up();
        }
        __syncwarp();
    } else if (warp >= WM_DQ + 2) {
        // ---- products: a warp for each tile, so that one's waits lie under the other's MMAs ----
        const int i = warp - (WM_DQ + 2);
        const uint32_t idesc = (1u << 4) | ((uint32_t)(dcols >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        const uint32_t xd = wm_desc(smem_u32(x_s)), half = (uint32_t)(p.nt * 128) >> 4;
        Ring ra, rx;
        int fold = FOLD ? i * APART : 0, used = 0;   // steps in the accumulator (the tiles in turn); times it was handed over
        bool fresh = true;                     // it starts anew
        bool ok = true;
        for (int s = 0; s < n; ++s, ra.next(p.sa)) {
            const uint32_t d = dt + (uint32_t)(i * dcols);
            if (FOLD && fresh && used > 0) ok = mbar_wait(&d_empty[i], (uint32_t)(used - 1) & 1u);
            ok = ok && mbar_wait(&x_full[rx.slot], rx.odd) && mbar_wait(&a_full[ra.slot], ra.odd);
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_after();
            const uint32_t a = at0 + (uint32_t)(ra.slot * AC + (WIDE ? 0 : i * 64));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (P == 2 && h == 1) {
                    ok = mbar_wait(&x_full[rx.slot], rx.odd);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_after();
                }
                const uint32_t x = xd + (uint32_t)(rx.slot * (xbytes >> 4));
                // B: half h of the stage, or (P == 2) a stage of 64 columns, both parts, WIDE: of a block of tokens
                mma_64(d, a + (uint32_t)(h * 32), x + (P == 1 ? h * half : WIDE ? i * P * half : 0u), idesc, fresh && h == 0 ? 0u : 1u);
                if (P == 2 || h == 1) {
                    commit(&x_empty[rx.slot]);
                    rx.next(p.sx);
                }
            }
            if (!ok) break;                    // the same for all lanes
            commit(&a_empty[ra.slot]);
            fresh = (FOLD && ++fold == WM_FOLD) || s + 1 == n;
            if (fresh) {
                commit(&d_full[i]);
                ++used;
                fold = 0;
            }
        }
        // no product may still read shared memory or TMEM when the CTA frees them, also where a wait gave up before its end
        commit(&done[i]);
        ok = mbar_wait(&done[i], 0u) && ok;
        if (!__all_sync(0xffffffffu, ok) && lane == 0) give_up();
        __syncwarp();
    } else {
        // ---- weights ----
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane;   // TMEM lane = tile row
        // the accumulator that the warpgroup takes: of its tile, or (WIDE) of a block of tokens, and then it makes the weights
        // of every other step; half of the step's columns
        const int mat = wg >> 1, h = wg & 1;
        const bool second = WIDE ? r >= 64 : mat == 1;          // GLU: the row is of the up matrix
        const int own = WIDE ? mat : 0;                         // its first step
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        // the rows' powers of two: a warp takes 16 rows, its lanes the scales of a row
        {
            const int g0 = s0 * (128 / G), g1 = min(spitch, s1 * (128 / G));
            constexpr int EACH_WARP = WIDE ? 8 : 16;            // rows of a warp
            const int i = WIDE ? 0 : warp >> 3;
            const bool up_rows = GLU && (WIDE ? warp >= 8 : i == 1);
            const int first = row0 + (GLU ? (WIDE && up_rows ? -64 : 0) : i * 128);
            const unsigned short* base = reinterpret_cast<const unsigned short*>(p.scales[GLU ? up_rows : i]);
#pragma unroll
            for (int j = 0; j < EACH_WARP; ++j) {
                const int rr = (WIDE ? warp : warp & 7) * EACH_WARP + j;
                uint32_t top = 0;
                if (first + rr < p.N) {
                    const unsigned short* s = base + (size_t)(first + rr) * spitch;
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
        const int nn = row0 + (WIDE ? (GLU ? r & 63 : r) : (GLU ? 0 : mat * 128) + r);   // this thread's row of its matrix
        const bool in = nn < p.N;
        const float up = row_up(row_e[WIDE ? 0 : mat][r]), down = row_down(row_e[WIDE ? 0 : mat][r]);
        const unsigned short* sp = reinterpret_cast<const unsigned short*>(p.scales[GLU ? second : WIDE ? 0 : mat]) + (size_t)(in ? nn : 0) * spitch;
        // eight scales of the row at a time, the next eight under way
        constexpr int WIN = 8 * G / 128;       // steps of eight groups
        uint4 sw = make_uint4(0u, 0u, 0u, 0u), sn = sw;
        int left = 0;                          // steps that sw still serves
        auto load_win = [&](int w) { return w * 8 < spitch ? __ldg(reinterpret_cast<const uint4*>(sp) + w) : make_uint4(0u, 0u, 0u, 0u); };
        if (p.wide) {
            sw = load_win((s0 + own) / WIN);
            sn = load_win((s0 + own) / WIN + 1);
            left = WIN - (s0 + own) % WIN;
        }
        // two parts: the sums of 32 tokens of this thread's row; tokens 32 h .. 32 h + 31 of tile `mat`
        float acc[FOLD ? 32 : 1];
#pragma unroll
        for (int e = 0; e < (FOLD ? 32 : 1); ++e) acc[e] = 0.f;
        int folded = 0;                        // times the tile's accumulator was taken
        auto fold_in = [&]() -> bool {
            // a lane's wait may run out by itself: all of the warp read TMEM, or none
            if (!__all_sync(0xffffffffu, mbar_wait(&d_full[mat], (uint32_t)folded & 1u))) return false;
            fence_after();
            if (h * 32 < p.nt) {
#pragma unroll
                for (int part = 0; part < P; ++part) {
                    uint32_t v[32];
                    tmem_ld32(dt + lanes + (uint32_t)(mat * dcols + part * p.nt + h * 32), v);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int e = 0; e < (FOLD ? 32 : 1); ++e) {
                        asm volatile("" : "+r"(v[e]));
                        acc[e] += __uint_as_float(v[e]);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[mat]);
            ++folded;
            return true;
        };
        const W4Const kc;
        uint32_t sixteen;                      // 16 in both halves, the code's sign bit turned over
        asm volatile("mov.b32 %0, 0x4e004e00;" : "=r"(sixteen));
        const int swz = (r >> 1) & 3;
        const unsigned char* row = codes_s + (WIDE ? 0 : mat * (CODES / 2)) + r * 64;
        const int c0 = ((2 * h) ^ swz) << 4, c1 = ((2 * h + 1) ^ swz) << 4;
        Ring rc, ra;
        bool ok = true;
        uint4 q0, q1;                          // a row's 32 bytes of codes
        auto read_codes = [&]() {
            ok = mbar_wait(&codes_full[rc.slot], rc.odd) && ok;
            q0 = *reinterpret_cast<const uint4*>(row + (size_t)rc.slot * CODES + c0);
            q1 = *reinterpret_cast<const uint4*>(row + (size_t)rc.slot * CODES + c1);
            rc.next(p.sc);
            if (WIDE) rc.next(p.sc);           // the rings' lengths are even, so a slot is always the same warpgroups'
        };
        if (WIDE && own) {
            rc.next(p.sc);
            ra.next(p.sa);
        }
        int now = WIDE ? rc.slot : 0;          // the slot that they came from
        if (!WIDE || own < n) read_codes();
        for (int s = own; s < n; s += EACH, ra.next(p.sa)) {
            const int step = s0 + s;
            uint32_t sc[NS];
            if (p.wide) {
                if (WIDE ? left <= 0 : left == 0) {
                    sw = sn;
                    sn = load_win(step / WIN + 1);
                    left = WIDE ? left + WIN : WIN;
                }
                left -= EACH;
#pragma unroll
                for (int c = 0; c < NS; ++c)
                    sc[c] = scale_pair(pick16(sw, (G == 128 ? step : G == 64 ? 2 * step + h : 4 * step + 2 * h + c) & 7), up);
            } else {
#pragma unroll
                for (int c = 0; c < NS; ++c) {
                    const int g = G == 128 ? step : G == 64 ? 2 * step + h : 4 * step + 2 * h + c;
                    sc[c] = g < spitch ? scale_pair(__ldg(sp + g), up) : 0u;
                }
            }
            const int codes_slot = now;
            now = rc.slot;
            const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
            if (s + EACH < n) read_codes();    // its next step's, under this one's arithmetic
            uint32_t a[32];
            {
                uint32_t f24[NS];
#pragma unroll
                for (int c = 0; c < NS; ++c) f24[c] = w4_hmul(sc[c], 0xce00ce00u);   // -24
#pragma unroll
                for (int c = 0; c < 8; ++c) unpack_scaled(w[c], kc, sixteen, sc[NS == 2 ? c >> 2 : 0], f24[NS == 2 ? c >> 2 : 0], a + c * 4);
            }
            if (s >= p.sa) ok = mbar_wait(&a_empty[ra.slot], ra.odd ^ 1u) && ok;
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_after();
            tm_st32(at0 + lanes + (uint32_t)(ra.slot * AC + (WIDE ? 0 : mat * 64) + h * 32), a);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&a_full[ra.slot]);
                // the codes have become weights, so they are read: at their load they were only asked for, and the next copy
                // could have come first
                mbar_arrive(&codes_empty[codes_slot]);
            }
            if (WIDE) ra.next(p.sa);
            // the accumulator is taken when the weights of the step behind its last are made: its products have had that long
            if (FOLD && s > 0 && (s + mat * APART) % WM_FOLD == 0) {
                ok = fold_in();
                if (!ok) break;                // the same for all lanes
            }
        }
        if (!__all_sync(0xffffffffu, ok) && lane == 0) give_up();

        // ---- epilogue ----
        pdl_wait();
        for (int i = tid; i < m; i += WM_DQ * 32) tok_f[i] = __ldcg(p.factor + tok0 + i);
        bool live = __all_sync(0xffffffffu, ok && !*ab);   // (another warp may set it between two lanes' reads)
        if (FOLD) {
            const int times = (n - 1 + mat * APART) / WM_FOLD + 1;
            while (live && folded < times) live = fold_in();
        } else if (live) {
            live = __all_sync(0xffffffffu, mbar_wait(&d_full[mat], 0u));
            fence_after();
        }
        if (!live && lane == 0) give_up();
        named_sync(1, WM_DQ * 32);
        live = __all_sync(0xffffffffu, !*ab);
        const int tb = WIDE ? mat * p.nt : 0, mh = WIDE ? min(p.nt, m - tb) : m;   // the accumulator's first token; its tokens
        // the smaller factor first: no step leaves fp32's range unless the result does
        auto sized = [&](float v, float b) { return v * fminf(down, b) * fmaxf(down, b); };
        // the results of up to 16 tokens from token c of the accumulator for output row nn: sums v (of the gate; then u of up)
        auto put16 = [&](int c, int count, float (&v)[16], float (&u)[16]) {
            if (GLU) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = w4_glu(p.act, v[e], u[e]);
            } else if (p.residual) {
                const size_t at = (size_t)(tok0 + tb + c) * p.residual_stride + nn;
                if (p.out_f32) {
                    const float* x = reinterpret_cast<const float*>(p.residual) + at;
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = e < count ? x[(size_t)e * p.residual_stride] : 0.f;
                } else {
                    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(p.residual) + at;
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = e < count ? __bfloat162float(x[(size_t)e * p.residual_stride]) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] += u[e];
            }
            const size_t at = (size_t)(tok0 + tb + c) * p.out_stride + nn;
            if (p.out_f32) {
                float* o = reinterpret_cast<float*>(p.out) + at;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < count) o[(size_t)e * p.out_stride] = v[e];
            } else {
                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < count) o[(size_t)e * p.out_stride] = __float2bfloat16_rn(v[e]);
            }
        };
        // Sums of 16 tokens from token c for this thread's row of its matrix.  Plain results go out from here; a gate's meet
        // the up's in shared memory, and a split's those of the other CTAs (in the rings: all copies have landed, all
        // weights are made, all products are done)
        constexpr int US = ROWS + 1;           // GLU: of a token's rows
        float* meet = reinterpret_cast<float*>(smem);            // [tokens][US]
        auto take16 = [&](int c, float (&v)[16]) {
            const int count = min(16, mh - c);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = e < count ? sized(v[e], tok_f[tb + c + e]) : 0.f;
            if (!WIDE && p.ks > 1) {
#pragma unroll
                for (int e = 0; e < 16; ++e) meet[(c + e) * WM_ROWS + mat * 128 + r] = v[e];
            } else if (GLU) {
                if (second) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) meet[(tb + c + e) * US + r % ROWS] = v[e];
                }
            } else if (in) {
                float u[16];
                put16(c, count, v, u);
            }
        };
        // P == 1: chunks of 16 tokens of a tile go to its two warpgroups in turn.  P == 2: they are in acc
        auto chunk = [&](int c, float (&v)[16]) {
            __syncwarp();                      // lanes without a row wrote nothing: all of the warp read TMEM together
            if (FOLD) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = c & 16 ? acc[FOLD ? 16 + e : 0] : acc[FOLD ? e : 0];
            } else {
                uint32_t d[16];
                tm_ld16(dt + lanes + (uint32_t)(mat * dcols + c), d);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    asm volatile("" : "+r"(d[e]));
                    v[e] = __uint_as_float(d[e]);
                }
            }
        };
        const int cfirst = FOLD ? h * 32 : h * 16, cstep = FOLD ? 16 : 32, cend = FOLD ? min(mh, h * 32 + 32) : mh;
        if (live) {
            for (int c = cfirst; c < cend; c += cstep) {
                float v[16];
                if (GLU && p.ks == 1 && !second) continue;       // up first
                chunk(c, v);
                take16(c, v);
            }
        }
        if (GLU && p.ks == 1) {
            named_sync(1, WM_DQ * 32);
            if (live && !second) {
                for (int c = cfirst; c < cend; c += cstep) {
                    float v[16], u[16];
                    const int count = min(16, mh - c);
                    chunk(c, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        v[e] = e < count ? sized(v[e], tok_f[tb + c + e]) : 0.f;
                        u[e] = meet[(tb + c + e) * US + r];
                    }
                    if (in) put16(c, count, v, u);
                }
            }
        }
    }
    if (!WIDE && p.ks > 1) {
        cluster_sync();
        // the tokens of this CTA's part, a row a thread: the sums of all CTAs of the cluster, in their order
        const float* sums = reinterpret_cast<const float*>(smem);
        constexpr int OUT = GLU ? 128 : 256;   // output rows
        const int r = tid % OUT, nn = row0 + r, t1 = (split + 1) * m / p.ks;
        if (tid < WM_DQ * 32 && nn < p.N) {
            for (int t = split * m / p.ks + tid / OUT; t < t1; t += WM_DQ * 32 / OUT) {
                float res = 0.f;
                if (!GLU && p.residual) res = w4_load1(p.residual, p.out_f32, (size_t)(tok0 + t) * p.residual_stride + nn);
                float v = 0.f, u = 0.f;
                for (int w = 0; w < p.ks; ++w) {
                    v += ld_cluster(sums + t * WM_ROWS + r, w);
                    if (GLU) u += ld_cluster(sums + t * WM_ROWS + 128 + r, w);
                }
                w4_store1(p.out, p.out_f32, (size_t)(tok0 + t) * p.out_stride + nn, GLU ? w4_glu(p.act, v, u) : v + res);
            }
        }
        cluster_sync();                        // until the others have read this CTA's sums
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
const void* gemm_kernel(int P, bool glu, bool wide) {
    if (wide) return glu ? (const void*)&k_w4_gemm<G, 2, true, true> : (const void*)&k_w4_gemm<G, 2, false, true>;
    if (P == 1) return glu ? (const void*)&k_w4_gemm<G, 1, true, false> : (const void*)&k_w4_gemm<G, 1, false, false>;
    return glu ? (const void*)&k_w4_gemm<G, 2, true, false> : (const void*)&k_w4_gemm<G, 2, false, false>;
}

const void* kernel_of(const W4Gemm& g) {
    const int P = g.parts;
    switch (g.c.group()) {
        case 32: return gemm_kernel<32>(P, g.c.glu, g.wide);
        case 64: return gemm_kernel<64>(P, g.c.glu, g.wide);
        default: return gemm_kernel<128>(P, g.c.glu, g.wide);
    }
}

int round_up(int v, int to) { return (v + to - 1) / to * to; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

cudaError_t w4_gemm_plan(W4Gemm* g, int num_sms) {
    const W4Call& c = g->c;
    const int rows = wm_rows(c.glu, false);
    const int tiles = (c.n() + rows - 1) / rows, steps = (c.k() + 127) / 128;
    // One part is not folded: 128 tokens' sums are twice the registers that a thread has for them.  What the tensor cores cut off
    // adds up over an accumulator's columns, at most 2^-23 of the sums for each 16.  Up to WM_UNFOLDED of them that is 2^-12, an
    // eighth of a bf16 result's half step (measured: 4e-5 of the whole); clusters keep to it where there are more columns.  An fp32
    // result shows it, so there bf16 activations take two parts, the second of zeros, and are folded: 893 us in place of 424 (4095
    // tokens, 14336 -> 4096), 50 in place of 36 (40 tokens)
    const int P = g->parts = c.parts() == 2 || c.out_f32 || steps > 8 * WM_UNFOLDED / 128 ? 2 : 1;
    // Tokens of a tile and CTAs along k: the least time of the longest CTA, in clocks.  A step takes the tensor cores 8
    // clocks a token and part, or the making and handing over of its weights 900; a CTA starts and ends in about 7000,
    // and a split adds the joining of its sums
    double best = -1.0;
    const int least = (c.tokens + wm_tokens(P) - 1) / wm_tokens(P);
    for (int blocks = least; blocks <= least + 8; ++blocks) {
        const int nt = round_up((c.tokens + blocks - 1) / blocks, 16), used = (c.tokens + nt - 1) / nt;
        for (int ks = 1; ks <= 8; ks *= 2) {
            if (ks > 1 && steps / ks < 2) break;
            if (P == 1 && (steps + ks - 1) / ks > WM_UNFOLDED / 128) continue;
            const long long places = ks == 1 ? num_sms : w4_clusters(ks, num_sms);
            const double waves = (double)(((long long)tiles * used + places - 1) / places);
            const double step = 8.0 * nt * P > 900.0 ? 8.0 * nt * P : 900.0;
            const double t = waves * ((double)((steps + ks - 1) / ks) * step + 7000.0 + 16.0 * nt) + (ks > 1 ? 2000.0 + 8.0 * nt : 0.0);
            if (best < 0.0 || t < best) {
                best = t;
                g->nt = nt;
                g->ks = ks;
            }
        }
        if (nt <= 16) break;
    }
    // Two parts: with one row tile and two blocks of tokens a CTA makes half the weights for as many products, and a
    // step takes 0.8 of the time; but it has no split along k, and the tiles have to fill the card. 1000 tokens, gate and up
    // 14336 x 4096, take 513 us against 607, 1024 tokens 4096 x 4096 82 against 102, 330 45 against 62; 520 tokens 14336 -> 4096
    // would be two waves half full, 250 against 170. With one part it gains nothing: 4095 tokens 14336 -> 4096 took 453 against 442
    if (P == 2 && c.tokens > wm_tokens(P)) {
        const int two = 2 * wm_tokens(P), few = (c.tokens + two - 1) / two;
        const int wide = (c.n() + wm_rows(c.glu, true) - 1) / wm_rows(c.glu, true);
        for (int blocks = few; blocks <= few + 8; ++blocks) {
            const int nt = round_up((c.tokens + 2 * blocks - 1) / (2 * blocks), 16), used = (c.tokens + 2 * nt - 1) / (2 * nt);
            const double waves = (double)(((long long)wide * used + num_sms - 1) / num_sms);
            const double step = 16.0 * nt > 900.0 ? 16.0 * nt : 900.0;
            const double t = waves * (0.8 * (double)steps * step + 7000.0 + 32.0 * nt);
            if (t < best) {
                best = t;
                g->nt = nt;
                g->ks = 1;
                g->wide = true;
            }
            if (nt <= 16) break;
        }
    }
    g->kp = round_up(c.k(), 64);
    g->steps = steps;
    const void* fn = kernel_of(*g);
    static OncePerDevice once[3][3][2];
    return once[c.group() == 32 ? 0 : c.group() == 64 ? 1 : 2][g->wide ? 2 : P - 1][c.glu].run([&] { return raise_smem_cap(fn); });
}

size_t w4_gemm_bytes(const W4Gemm& g) {
    const W4Call& c = g.c;
    const int P = g.parts;
    return round256((size_t)P * c.tokens * g.kp * 2) + round256((size_t)c.tokens * 4);
}

cudaError_t w4_gemm_launch(const W4Gemm& g, cudaStream_t s) {
    const W4Call& c = g.c;
    const int P = g.parts, mats = c.glu ? 2 : 1;
    __half* parts = (__half*)g.ws;
    float* factor = (float*)((char*)g.ws + round256((size_t)P * c.tokens * g.kp * 2));
    WmParams p{};
    for (int i = 0; i < 2; ++i) {
        const W4Matrix& w = c.w[i < mats ? i : 0];
        if (!encode(&p.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.n, w.k / 2, w.k / 2, 64, g.wide && c.glu ? 64 : 128,
                    CU_TENSOR_MAP_SWIZZLE_64B))
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
    p.steps = g.steps;
    p.act = c.act;
    p.out_f32 = c.out_f32;
    p.wide = (c.k() / c.group()) % 8 == 0 && ((uintptr_t)p.scales[0] & 15) == 0 && ((uintptr_t)p.scales[1] & 15) == 0;
    p.err = c.err;
    // the rings: four stages of codes at least (behind the last step they also hold a tile's up sums), then activations
    const int xb = wm_stage(g.wide, g.nt), cb = wm_codes(g.wide);
    p.sx = (WM_SMEM - 5 * cb) / xb;
    if (p.sx > WM_MAX_SX) p.sx = WM_MAX_SX;
    p.sc = (WM_SMEM - p.sx * xb) / cb;
    if (p.sc > WM_MAX_SC) p.sc = WM_MAX_SC;
    p.sa = (512 - 2 * g.nt * P) / (g.wide ? 64 : 128);
    if (p.sa > WM_MAX_SA) p.sa = WM_MAX_SA;
    if (g.wide) {                              // even: a warpgroup makes every other step's weights
        p.sc &= ~1;
        p.sa &= ~1;
    }
    if (p.sx < 2 || p.sc < 4 || p.sa < 2) return cudaErrorInvalidValue;

    if (P == 1)
        k_w4_split<1><<<c.tokens, WS_THREADS, 0, s>>>(c.x, c.x_stride, c.x_f32, c.gain, c.gain_f32, c.eps, c.k(), g.kp, c.tokens, parts, factor);
    else
        k_w4_split<2><<<c.tokens, WS_THREADS, 0, s>>>(c.x, c.x_stride, c.x_f32, c.gain, c.gain_f32, c.eps, c.k(), g.kp, c.tokens, parts, factor);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int rows = wm_rows(c.glu, g.wide), block = g.wide ? 2 * g.nt : g.nt;
    cfg.gridDim = dim3((c.n() + rows - 1) / rows * g.ks, (c.tokens + block - 1) / block);
    cfg.blockDim = dim3(WM_THREADS);
    cfg.dynamicSmemBytes = (size_t)p.sx * xb + (size_t)p.sc * cb + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];   // starts while k_w4_split runs: codes and scales do not depend on it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.ks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = g.ks > 1 ? 2 : 1;
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, kernel_of(g), args);
}

}  // namespace gd
