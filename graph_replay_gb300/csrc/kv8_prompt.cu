// kv8_prompt.cu -- attention over the 8-bit K/V cache for prompts and chunks
// (more than 16 query rows of a K/V head) on the 5th-generation tensor cores.
//
// The query rows of a K/V head are (token, query head of the group), tokens
// first: a tile of 128 holds all G heads of 128 / G tokens, so the heads share
// every K/V tile and little of a tile lies above the causal diagonal.  Any G
// works: a tile may begin inside a token.  A CTA has two query tiles, and per 64
// positions (the one K/V tile that both read):
//   convert   four warps for the even tiles and four for the odd read the e4m3
//             bytes (the pages' own order) two tiles ahead, turn K into f16 and V
//             times its scale into bf16 -- both exact -- and store them as
//             128-byte-swizzled operand tiles in a ring; page ids and scales are
//             read a batch of tiles earlier.  V's NaN become 0 (below)
//   S = Q K^T tcgen05.mma kind::f16, A = Q, B = K, D in TMEM; two S buffers for
//             each query tile, so the product runs a tile ahead of the softmax
//   softmax   a thread owns a row: scores times K's scale, running maximum kept
//             within 2^8, weights as two bf16 parts (16 bits and more, with fp32's
//             range) back into TMEM over the scores they came from
//   O += P V  A = P from TMEM, B = V read MN-major, in bf16
// The largest weight may belong to a position whose V is 0 in a dim, and V's scales
// may lie far apart, so small weights have to keep their digits: f16 holds 20 bits
// below the largest, bf16 what fp32 does.  It has 8 bits where f16 has 11, hence two
// parts for a weight, and that is what bf16 prompts pay for it (8191 tokens: one
// f16 part 540 us, two bf16 parts 620; the second product itself costs 15 of them;
// scores rounded before the maximum is subtracted 20 more).
// 64 positions rather than 128: with 128 there is room for one S a query tile,
// and product and softmax wait for one another (8191 tokens: 682 -> 633 us with
// the change, although S = Q K^T of 64 columns reads Q from shared memory twice as
// often and takes 48 cycles where 32 would do).
// With fp32 q, q enters as two f16 parts and the weights as three bf16 parts (two:
// relative error 2.6e-6, three: 1.2e-6).  Two parts of P lie side by side over their
// scores, the third in TMEM (64 dims) or in shared memory (128: TMEM is full).  The
// tensor core's accumulator cuts off what it adds, so O is folded into memory in
// rounded sums every KP_FOLD tiles.
//
// Each query tile has its own issuing warp: a wait costs its trip through a busy
// shared memory (about 250 cycles) even where nothing is left to wait for, and
// with one warp for both tiles those trips, not the products, filled its time
// (8191 tokens: 602 -> 543 us; K's and V's waits as one: 539).
//
// Bound, measured: 8191 tokens 640 us, 45 % of the measured bf16 rate; 2 x 64 fp32
// tokens over 32k 111 us with 64 dims, 195 with 128.  The chain of a tile's steps binds it -- P to S of the
// tile after the next to P again -- and the hand-overs in it.  With one f16 part a
// weight (540 us) a K/V tile took about 2200 cycles, of which the tensor core needed
// 1280 (now 1790) and a softmax warp 1700.  Leaving out half of the MMAs, the
// exponentials and the maximum, or the loads and conversions, brought some 20 us
// each, all of them 145.  What did not help then: S two tiles ahead, right behind
// P V (544); 16 softmax warps, two threads a row (572); one arrival a warp instead
// of a thread; other shares of the registers.
// V's conversion is eight instructions for two values where f16 took one.  With K
// and V in four warps each, V's warps, which also wait for their loads, could not
// follow the tiles (800 us); with a tile's K and V in the same warps, every other
// tile each, they do.
//
// Few tiles and many positions: the positions of a tile are split over several
// CTAs (a host rule on sizes) and joined by a second kernel in split order.
// Results leave through shared memory, row by row.
//
// NaN: 0 * NaN is NaN inside an MMA, so a NaN in V that one row of a tile sees
// would reach the rows that do not.  Therefore V's NaN never enter the product;
// a tile that held one is marked, and at the end each row looks through the
// marked tiles for NaN that it sees.  Positions that nobody sees are stored as
// zeros.  Masked scores are replaced, never multiplied.
#include <limits.h>
#include <type_traits>
#include "kv8.cuh"
#include "mma_helpers.cuh"

namespace gd {

namespace {

constexpr int KP_ROWS = 128;              // query rows of a tile: TMEM lanes
constexpr int KP_KEYS = 64;               // positions of a tile
// 8 softmax warps, 8 that convert K and V, 2 that issue MMAs and 2 that only pad their warpgroup
constexpr int KP_CONV_WARP = 8, KP_MMA_WARP = 16, KP_THREADS = 20 * 32;
// registers a thread by role (setmaxnreg): 640 threads x 96 at launch = 256 x 120 + 256 x 88 + 128 x 64
constexpr int KP_REGS_SOFTMAX = 120, KP_REGS_CONV = 88, KP_REGS_MMA = 64;
constexpr int KP_QPANEL = KP_ROWS * 128, KP_PANEL = KP_KEYS * 128;   // bytes of 64 dims of a query tile, of a K or V tile
constexpr float KP_SLACK = 8.f, KP_SHIFT = -8.f;   // log2: maximum may lag; weights carry 2^-8, so none is above 1
// fp32 q: tiles between two folds of O into memory (64 tokens over 32k, relative error and time: 12 2.2e-6, 101 us; 8
// 1.6e-6, 106; 6 1.2e-6, 109, before scores were rounded first.  fp32 sums in the plain order: 2.9e-6, but 0.9e-6 over 2000 positions)
constexpr int KP_FOLD = 6;
constexpr int KP_META = 8;                // tiles whose scales are held
constexpr int KP_GROUPS = KP_KEYS / 16, KP_BATCH = 32 / KP_GROUPS;   // 16-position groups of a tile; tiles that a warp's lanes know of
constexpr int KP_MARKS = 32;              // words of marks: tile i has bit i % (32 * KP_MARKS)

template <int HD, bool FINE>
struct KpLayout {
    static constexpr int PARTS = FINE ? 2 : 1;
    static constexpr int QTILE = HD / 64 * KP_QPANEL, TILE = HD / 64 * KP_PANEL;   // bytes of f16 operand tiles
    static constexpr int SLOTS = HD == 128 && FINE ? 4 : 8;                         // K and V tiles in turn
    // fp32 q, the weights' third parts: TMEM has room for them beside 64 dims, else a tile in shared memory
    static constexpr bool THIRD_TMEM = FINE && HD == 64, THIRD_SMEM = FINE && HD == 128;
    static constexpr int PTILE = THIRD_SMEM ? KP_QPANEL : 0;
    static constexpr int Q = 0, KV = 2 * PARTS * QTILE, P3 = KV + SLOTS * TILE, BYTES = P3 + 2 * PTILE;
    // TMEM columns: S of query tile x, buffer b at 128 x + 64 b (P lies over it), O of query tile x at 256 + HD x, third
    // parts at 384 + 64 x + 32 b
    static constexpr int O = 256, THIRD = 384;
};
template <int HD, bool FINE>
constexpr int kp_smem() { return KpLayout<HD, FINE>::BYTES + 1024; }

// byte offset of 16-byte chunk c of row r in a panel (128-byte swizzle)
__device__ __forceinline__ uint32_t kp_sw(int r, int c) {
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}
// shared-memory descriptor of 128-byte-swizzled tiles: the low word holds the address and the stride
// between panels (both in 16 bytes), the high word is the same for all
__device__ __forceinline__ uint32_t kp_desc(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t KP_DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
// kind::f16, fp32 D; Q K^T: f16 A and B, both K-major; P V: bf16 A and B, B MN-major
constexpr uint32_t kp_idesc(int N, bool pv) {
    return (1u << 4) | (pv ? 1u << 7 | 1u << 10 | 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(KP_ROWS >> 4) << 24);
}
// One thread issues every MMA of a query tile, so what it does for each lies on the tensor core's path.  The whole warp
// runs the issuing code, every lane has the operands, and each run of four MMAs (four steps of 16) or commit elects the
// lane that issues it.

// D (+)= A B over 64 dims, both tiles in shared memory.  acc 0: D starts anew
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred e, p, t;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
                 " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n add.u64 x, x, 2;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n add.u64 x, x, 2;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n add.u64 x, x, 2;\n add.u64 y, y, 2;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(KP_DESC_HI),
                 "r"(idesc), "r"(acc)
                 : "memory");
}
// D (+)= A B over 64 positions, A in TMEM (8 columns a step), B's rows 128 bytes apart
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred e, p, t;\n .reg .b64 y;\n .reg .b32 a;\n setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
                 " mov.b32 a, %1;\n mov.b64 y, {%2, %3};\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, p;\n add.u32 a, a, 8;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n add.u32 a, a, 8;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, t;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(KP_DESC_HI),
                 "r"(idesc), "r"(acc)
                 : "memory");
}
// the same with A in shared memory
__device__ __forceinline__ void mma_st4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred e, p, t;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
                 " mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n add.u64 x, x, 2;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n add.u64 x, x, 2;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n add.u64 x, x, 2;\n add.u64 y, y, 128;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(KP_DESC_HI),
                 "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void kp_commit(uint64_t* bar) {
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t (&r)[32]) {
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
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t pack_b2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 values times 2^e as packed bf16 pairs, exact: 4 significant bits, fp32's exponents (an e above 118, which is
// flagged, would make an infinity of 448, and NaN with a weight of 0).  A byte s eeee mmm, moved to s 0000 eeee mmm 0000, is the bf16 of
// its value times 2^-120, subnormals too.  2^(e + 120) passes the range, so it is two factors
struct KpScale {
    __nv_bfloat162 a, b;
    __device__ __forceinline__ explicit KpScale(int e) {
        const int n = min(e, 118) + 120, h = n >> 1;
        a = __float2bfloat162_rn(pow2i(h));
        b = __float2bfloat162_rn(pow2i(n - h));
    }
    __device__ __forceinline__ uint32_t two(uint32_t x) const {   // bytes in the high halves
        const uint32_t w = (x & 0x7F007F00u) >> 4 | (x & 0x80008000u);
        const __nv_bfloat162 y = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), a), b);
        return *reinterpret_cast<const uint32_t*>(&y);
    }
    __device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) const {
        lo = two(__byte_perm(w, 0u, 0x1404));
        hi = two(__byte_perm(w, 0u, 0x3424));
    }
};
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// what the scores of 16 positions of a tile need
struct __align__(8) KpMeta {
    float kf, add;   // 2^K exponent; 0, or -inf where nothing is held
};

// every warp of the CTA, each from its own role
__device__ __forceinline__ void cta_meet() { asm volatile("bar.sync 0;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// two fp32 at once
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Whether the phase with this parity completes within about KP_WAIT_NS (the thread sleeps meanwhile)
constexpr uint32_t KP_WAIT_NS = 20000;
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(KP_WAIT_NS)
        : "memory");
    return ok != 0;
}
// A whole warp waits, bounded (about two seconds; FAULT_WAIT then).  One lane polls, and sleeps between polls: two
// fifths of the instructions were those of spinning warps (they filled idle slots: the time hardly changed).  False: this wait has given up, or another role has
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* aborted, unsigned* err) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;   // mostly it is done already
    bool go = true;
    if ((threadIdx.x & 31) == 0) {
        const long long t0 = clock64();
        while (!sleep_wait(bar, parity)) {
            if (!*aborted && clock64() - t0 < 4000000000ll) continue;
            go = false;
            *aborted = 1;
            atomicOr(err, FAULT_WAIT);
            break;
        }
    }
    return __all_sync(0xffffffffu, go);
}

// what turns a product into a score (log2); never 0, which would make NaN of a masked -inf
__device__ __forceinline__ float kp_mul(float fac, float kf) { return fmaxf(fac * kf, 1.17549435e-38f); }

// floats of the splits' parts (O, then M and l of each), up to a multiple of 16 bytes
__host__ __device__ __forceinline__ size_t kp_part_floats(int splits, size_t all_rows, int hd) {
    return splits == 1 ? 0 : (splits * all_rows * (hd + 2) + 3) / 4 * 4;
}

// the tiles of a CTA's rows: `sink` first ones, `gap` that no row sees, the rest
struct KpTiles {
    int n, sink, gap, end, low;   // tiles; first position behind; first position of the earliest window
};
__device__ __forceinline__ KpTiles kp_tiles(int pmin, int pmax, int window, int sinks) {
    KpTiles t{};
    t.end = max(pmax + 1, 0);
    t.low = (int)max((long long)max(pmin, 0) - window + 1, 0ll);
    const int end = (t.end + KP_KEYS - 1) / KP_KEYS, low = t.low / KP_KEYS;
    const int sink = (min(sinks, t.end) + KP_KEYS - 1) / KP_KEYS;
    if (sink >= low) {
        t.n = t.sink = end;
    } else {
        t.n = sink + end - low;
        t.sink = sink;
        t.gap = low - sink;
    }
    return t;
}

// The parts that the tiles of a CTA's rows are split into, of at most `splits` CTAs: at least 8 tiles each, since a
// CTA's beginning and end cost as much as two and the parts have to be joined
__host__ __device__ __forceinline__ int kp_parts(int tiles, int splits) {
    const int n = (tiles + 7) / 8;
    return n < 1 ? 1 : n < splits ? n : splits;
}

// grid (Hkv * query tiles, rows * splits)
template <int HD, bool FINE>
__global__ void __launch_bounds__(KP_THREADS, 1) k_kv8_prompt(const Kv8Attend p, int most) {
    using T = typename std::conditional<FINE, float, __nv_bfloat16>::type;
    using LY = KpLayout<HD, FINE>;
    constexpr int NQ = 2, SLOTS = LY::SLOTS;
    extern __shared__ __align__(1024) unsigned char kp_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(kp_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t kv_full[SLOTS], kv_empty[SLOTS], s_full[4], p_full[4], pv_done[4], meta_full[KP_META], all_done[2];
    __shared__ KpMeta meta[KP_META][KP_GROUPS];
    __shared__ float fac_s[NQ * KP_ROWS];
    __shared__ uint32_t marks[KP_MARKS];
    __shared__ uint32_t tmem;
    __shared__ int aborted, marked;

    pdl_wait();
    const Kv8Cache& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, h = (gridDim.x - 1 - blockIdx.x) % c.Hkv, r = blockIdx.y / most, sp = blockIdx.y % most;
    Kv8Row row;
    if (!kv8_row(p.b, c.ppr * c.page, r, &row)) return;
    const int rows_q = row.n * G;   // max_new * n_heads <= 2^30
    // tiles with the most positions first
    const int base = (int)((gridDim.x - 1 - blockIdx.x) / c.Hkv) * (NQ * KP_ROWS);
    if (base >= rows_q) return;
    const int nact = base + KP_ROWS < rows_q ? 2 : 1;   // query tiles in use
    const int p0 = row.len - row.n;
    const int tok0 = p.by_group.of(base), tok1 = p.by_group.of(min(base + NQ * KP_ROWS, rows_q) - 1);
    const KpTiles tl = kp_tiles(p0 + tok0, p0 + tok1, p.window, p.sinks);
    const int splits = kp_parts(tl.n, most);   // of this CTA's rows
    if (sp >= splits) return;
    const int i0 = (int)((long long)tl.n * sp / splits), i1 = (int)((long long)tl.n * (sp + 1) / splits);
    const int ntiles = i1 - i0;
    auto key0 = [&](int i) { return (i < tl.sink ? i : i + tl.gap) * KP_KEYS; };

    // ---- setup: Q as f16 tiles, each row brought to [2^14, 2^15) by a power of two ----
    if (ntiles > 0) {
        constexpr int LPR = HD / 8;   // lanes of a row, 8 dims each
        for (int x = tid; x < NQ * KP_ROWS * LPR; x += KP_THREADS) {   // a whole warp keeps whole rows: KP_THREADS % 32 == 0
            const int m = x / LPR, ch = x % LPR;
            float v[8];
            if (base + m < rows_q) {
                const int tk = p.by_group.of(base + m), hq = h * G + base + m - tk * G;
                const T* src = static_cast<const T*>(p.q) + (row.t0 + tk) * p.q_stride + hq * HD + ch * 8;
                if constexpr (FINE) {
                    const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                } else {
                    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(src)), v);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
            }
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
            const unsigned grp = LPR == 16 ? 0xFFFFu << (lane & 16) : 0xFFu << (lane & 24);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(grp, top, o));
            const int ex = min(max(268 - (int)(__float_as_uint(top) >> 23), 1), 254);
            const float up = __int_as_float(ex << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = v[2 * e] * up, b = v[2 * e + 1] * up;
                hi[e] = pack_h2(a, b);
                const float2 f = unpack_h2(hi[e]);
                lo[e] = pack_h2(a - f.x, b - f.y);
            }
            unsigned char* q = sm + LY::Q + (m / KP_ROWS) * (LY::PARTS * LY::QTILE) + (ch / 8) * KP_QPANEL + kp_sw(m % KP_ROWS, ch % 8);
            *reinterpret_cast<uint4*>(q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (FINE) *reinterpret_cast<uint4*>(q + LY::QTILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (ch == 0) fac_s[m] = p.scale * KV8_LOG2E / up;
        }
    }
    if (warp == KP_MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&kv_full[s], 128);
            mbar_init(&kv_empty[s], nact);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[2 * x], 1);
            mbar_init(&s_full[2 * x + 1], 1);
            mbar_init(&p_full[2 * x], 128);
            mbar_init(&p_full[2 * x + 1], 128);
            mbar_init(&pv_done[2 * x], 1);
            mbar_init(&pv_done[2 * x + 1], 1);
            mbar_init(&all_done[x], 1);
        }
        for (int x = 0; x < KP_META; ++x) mbar_init(&meta_full[x], 1);
        aborted = 0;
        marked = 0;
        mbar_fence_init();
    }
    if (tid < KP_MARKS) marks[tid] = 0u;
    fence_proxy_async_smem();   // Q's generic writes before the tensor core reads them
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t dt = tmem;
    volatile int* ab = &aborted;
    auto give_up = [&]() {
        *ab = 1;
        atomicOr(p.b.err, FAULT_WAIT);
    };
    if (warp >= KP_CONV_WARP && warp < KP_MMA_WARP) {
        // ---- K and V tiles: global e4m3 -> operand tiles, K in f16, V times its scale in bf16 ----
        regs_down<KP_REGS_CONV>();
        constexpr int KU = KP_KEYS / 32, LOADS = KU * (HD / 64);   // 16-byte loads of a thread: keys quad + 32 u of each panel
        const int grp = (warp - KP_CONV_WARP) / 4, ct = tid & 127, quad = ct >> 2, q4 = ct & 3;   // four warps have the even tiles, four the odd
        const size_t in_group = (size_t)(quad & 15) * HD + q4 * 16;
        // KP_BATCH tiles at a time, lane KP_GROUPS i + g knows of the 16 positions g of tile i: where they begin in the pool, in
        // 16 rows (-1: nowhere), and their scale bytes.  Both are read a batch ahead -- the page ids first, the
        // scales two tiles later -- so that no tile waits for them
        const int nb = c.page / c.block;
        int at = -1, at_next = -1, scales = 0, scales_next = 0;   // K's byte, V's << 8
        long long scale_at = 0;
        auto pages_ahead = [&](int j) {    // the batch that begins with tile j of this CTA
            const int i = i0 + j + lane / KP_GROUPS;
            at_next = -1;
            if (i >= i1) return;
            const int kb = key0(i) + 16 * (lane % KP_GROUPS);
            if (kb >= tl.end || (kb + 15 < tl.low && kb >= p.sinks)) return;
            const int slot = kb / c.page, off = kb - slot * c.page, page = kv8_page(c, p.b.err, r, slot);
            if (page < 0) return;
            const long long head = (long long)page * c.Hkv + h;
            at_next = (int)((head * c.page + off) / 16);
            scale_at = head * nb + off / c.block;
        };
        auto scales_ahead = [&]() {
            if (at_next >= 0) scales_next = (int)c.ks[scale_at] | (int)c.vs[scale_at] << 8;
        };
        auto check_scales = [&]() {   // of the batch held
            if (at >= 0 && !(kv8_scale_ok(scales & 255) && kv8_scale_ok(scales >> 8))) atomicOr(p.b.err, FAULT_SCALE);
        };
        uint4 k[LOADS], v[LOADS];
        auto load = [&](int j) {   // tile j, in the batch of `at`
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const int b = __shfl_sync(0xffffffffu, at, j % KP_BATCH * KP_GROUPS + 2 * u + (quad >> 4));
                const size_t from = (size_t)b * (16 * HD) + in_group;
#pragma unroll
                for (int n = 0; n < HD / 64; ++n) {
                    k[n * KU + u] = b >= 0 ? __ldg(reinterpret_cast<const uint4*>(c.k + from) + 4 * n) : make_uint4(0u, 0u, 0u, 0u);
                    v[n * KU + u] = b >= 0 ? __ldg(reinterpret_cast<const uint4*>(c.v + from) + 4 * n) : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        };
        auto slot = [&](int s) -> unsigned char* {   // null: the wait for it gave up
            if (s >= SLOTS && !warp_wait(&kv_empty[s % SLOTS], (uint32_t)(s / SLOTS - 1) & 1u, ab, p.b.err)) return nullptr;
            return sm + LY::KV + (s % SLOTS) * LY::TILE;
        };
        auto put = [&](unsigned char* tile, int u, int half, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
            *reinterpret_cast<uint4*>(tile + u / KU * KP_PANEL + kp_sw(quad + 32 * (u % KU), 2 * q4 + half)) = make_uint4(x, y, z, w);
        };
        if (ntiles > grp) {
            pages_ahead(0);
            scales_ahead();
            at = at_next;
            scales = scales_next;
            load(grp);
        }
        for (int j = grp; j < ntiles; j += 2) {
            const int in_batch = j % KP_BATCH;
            if (in_batch == grp) pages_ahead(j - grp + KP_BATCH);
            if (in_batch == 2 + grp) scales_ahead();
            unsigned char* tile = slot(2 * j);   // K and V tiles in turn
            if (!tile) break;
            if (ct < 32) {   // the last reader of this entry, the softmax of tile j - KP_META, is done: the ring is shorter
                if (lane / KP_GROUPS == in_batch)
                    meta[j % KP_META][lane % KP_GROUPS] = at >= 0 ? KpMeta{pow2i((scales & 255) - 127), 0.f} : KpMeta{1.f, -INFINITY};
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_full[j % KP_META]);
            }
#pragma unroll
            for (int u = 0; u < LOADS; ++u) {
                uint32_t a[4], b[4];
                e4m3x4_to_f16(k[u].x, a[0], a[1]);
                e4m3x4_to_f16(k[u].y, a[2], a[3]);
                e4m3x4_to_f16(k[u].z, b[0], b[1]);
                e4m3x4_to_f16(k[u].w, b[2], b[3]);
                put(tile, u, 0, a[0], a[1], a[2], a[3]);
                put(tile, u, 1, b[0], b[1], b[2], b[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&kv_full[2 * j % SLOTS]);
            // V's NaN stay out of the product; those at positions that a row of the CTA sees are marked
            uint32_t bad = 0u;
#pragma unroll
            for (int u = 0; u < LOADS; ++u) bad |= nan_bytes(v[u].x) | nan_bytes(v[u].y) | nan_bytes(v[u].z) | nan_bytes(v[u].w);
            if (bad) {
                bool seen = false;
#pragma unroll
                for (int u = 0; u < LOADS; ++u) {
                    const uint32_t n[4] = {nan_bytes(v[u].x), nan_bytes(v[u].y), nan_bytes(v[u].z), nan_bytes(v[u].w)};
                    const int key = key0(i0 + j) + quad + 32 * (u % KU);
                    if ((n[0] | n[1] | n[2] | n[3]) && key < tl.end && (key >= tl.low || key < p.sinks)) seen = true;
                    v[u].x &= ~((n[0] >> 7) * 0xFFu);
                    v[u].y &= ~((n[1] >> 7) * 0xFFu);
                    v[u].z &= ~((n[2] >> 7) * 0xFFu);
                    v[u].w &= ~((n[3] >> 7) * 0xFFu);
                }
                if (seen) {
                    atomicOr(&marks[(i0 + j) / 32 % KP_MARKS], 1u << ((i0 + j) & 31));
                    marked = 1;
                }
            }
            if (!(tile = slot(2 * j + 1))) break;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const KpScale s((__shfl_sync(0xffffffffu, scales, in_batch * KP_GROUPS + 2 * u + (quad >> 4)) >> 8) - 127);
#pragma unroll
                for (int n = 0; n < HD / 64; ++n) {
                    uint32_t a[4], b[4];
                    const uint4 w = v[n * KU + u];
                    s.widen(w.x, a[0], a[1]);
                    s.widen(w.y, a[2], a[3]);
                    s.widen(w.z, b[0], b[1]);
                    s.widen(w.w, b[2], b[3]);
                    put(tile, n * KU + u, 0, a[0], a[1], a[2], a[3]);
                    put(tile, n * KU + u, 1, b[0], b[1], b[2], b[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&kv_full[(2 * j + 1) % SLOTS]);
            if (in_batch == KP_BATCH - 2 + grp) {   // tile j + 2 lies in the next batch
                check_scales();
                at = at_next;
                scales = scales_next;
            }
            if (j + 2 < ntiles) load(j + 2);
        }
        check_scales();
        cta_meet();
    } else if (warp >= KP_MMA_WARP) {
        // ---- MMA issuers: a warp for each query tile, so that one's waits do not hold up the other's products ----
        regs_down<KP_REGS_MMA>();
        const int x = warp - KP_MMA_WARP;   // query tile
        if (x < nact && ntiles > 0) {
            constexpr uint32_t id_s = kp_idesc(KP_KEYS, false), id_o = kp_idesc(HD, true);
            const uint32_t dtu = __shfl_sync(0xffffffffu, dt, 0), xu = __shfl_sync(0xffffffffu, (uint32_t)x, 0);
            const int nt = __shfl_sync(0xffffffffu, ntiles, 0);
            const uint32_t qd = kp_desc(smem_u32(sm + LY::Q), 16) + xu * (LY::PARTS * LY::QTILE >> 4);
            const uint32_t kd = kp_desc(smem_u32(sm + LY::KV), 16), vd = kp_desc(smem_u32(sm + LY::KV), KP_PANEL);
            const uint32_t sd = dtu + 128 * xu, od = dtu + LY::O + HD * xu;
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                const bool there = warp_wait(bar, parity, ab, p.b.err);
                fence_after();
                return there;
            };
            auto qk = [&](int j) {   // S of tile j, into buffer j & 1
                const uint32_t kt = kd + (uint32_t)((2 * j) % SLOTS) * (LY::TILE >> 4), scol = sd + 64 * (j & 1);
                // q's second parts first: the accumulator cuts off what is added, relative to what it holds, and that is little yet
                if constexpr (FINE) {
#pragma unroll
                    for (int n = 0; n < HD / 64; ++n)
                        mma_ss4(scol, qd + (LY::QTILE >> 4) + n * (KP_QPANEL >> 4), kt + n * (KP_PANEL >> 4), id_s, n > 0);
                }
#pragma unroll
                for (int n = 0; n < HD / 64; ++n) mma_ss4(scol, qd + n * (KP_QPANEL >> 4), kt + n * (KP_PANEL >> 4), id_s, FINE || n > 0);
                kp_commit(&s_full[2 * xu + (j & 1)]);
            };
            auto pv = [&](int j) {
                const uint32_t vt = vd + (uint32_t)((2 * j + 1) % SLOTS) * (LY::TILE >> 4), pcol = sd + 64 * (j & 1);
                const uint32_t acc = (FINE ? j % KP_FOLD : j) > 0;
                if constexpr (LY::THIRD_TMEM) mma_ts4(od, dtu + LY::THIRD + 64 * xu + 32 * (j & 1), vt, id_o, acc);
                if constexpr (LY::THIRD_SMEM) mma_st4(od, kp_desc(smem_u32(sm + LY::P3), 16) + xu * (LY::PTILE >> 4), vt, id_o, acc);
                mma_ts4(od, pcol + 32, vt, id_o, FINE ? 1u : acc);
                mma_ts4(od, pcol, vt, id_o, 1u);
            };
            auto full = [&](int s) { return wait(&kv_full[s % SLOTS], (uint32_t)(s / SLOTS) & 1u); };
            bool ok = full(0);
            if (ok) {
                qk(0);
                kp_commit(&kv_empty[0]);
            }
            for (int j = 0; j < nt && ok; ++j) {
                const bool more = j + 1 < nt;
                const int sv = 2 * j + 1, sk = more ? 2 * j + 2 : sv;
                auto there = [&](int s) { return mbar_try_wait(&kv_full[s % SLOTS], (uint32_t)(s / SLOTS) & 1u); };
                // a wait costs a trip through a busy shared memory even where nothing is left to wait for: both at once
                if (__all_sync(0xffffffffu, there(sv) & there(sk))) fence_after();
                else if (!(ok = full(sv) && full(sk))) break;
                if (more) {
                    qk(j + 1);   // into the other buffer: its P has been multiplied, in order
                    kp_commit(&kv_empty[sk % SLOTS]);
                }
                if (!(ok = wait(&p_full[2 * xu + (j & 1)], (uint32_t)(j >> 1) & 1u))) break;
                pv(j);
                if (j + 2 >= nt) kp_commit(&pv_done[2 * xu + (j == nt - 1)]);
                kp_commit(&kv_empty[sv % SLOTS]);
            }
            // every MMA issued has finished before TMEM is released (also after a give-up)
            kp_commit(&all_done[xu]);
            if (lane == 0 && !mbar_wait(&all_done[xu], 0u)) give_up();
        }
        __syncwarp();
        cta_meet();
    } else {
        // ---- softmax: warp w reads TMEM lanes 32 (w % 4) + lane, the rows of query tile w / 4 ----
        regs_up<KP_REGS_SOFTMAX>();
        const int x = warp / 4, m = (warp & 3) * 32 + lane;
        const int mq = base + x * KP_ROWS + m;
        const bool live = x < nact && mq < rows_q;
        const int any = live ? mq : base, tk = p.by_group.of(any), hq = h * G + any - tk * G, pos = live ? p0 + tk : -1;
        const uint32_t lrow = dt + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ocol = lrow + LY::O + (uint32_t)(HD * x);
        float M = -INFINITY, l = 0.f;
        bool ok = true;
        const float fac = ntiles > 0 ? fac_s[x * KP_ROWS + m] : 0.f;
        // the positions of this query tile's rows
        const int xmin = p0 + p.by_group.of(base + x * KP_ROWS);
        const int xmax = p0 + p.by_group.of(min(base + (x + 1) * KP_ROWS, rows_q) - 1);
        const int lo = (int)max((long long)pos - p.window + 1, 0ll);   // this row sees [lo, pos] and [0, sinks)
        const size_t qrow = (size_t)(row.t0 + tk) * p.Hq + hq, all_rows = (size_t)p.b.total * p.Hq;
        T* dst = static_cast<T*>(p.out) + (row.t0 + tk) * p.out_stride + hq * HD;   // the result, or this split's part of it
        float* piece = p.ws + (sp * all_rows + qrow) * HD;
        // fp32 q: the tensor core cuts what it adds to its accumulator off, towards 0, and that shows after hundreds of
        // additions (7e-6 after 450).  So O is folded into memory every KP_FOLD tiles, in rounded sums: 16 bytes of
        // each row side by side, the rows of a CTA together (in the result's own rows a fold took 8 us)
        const size_t fold_tile = ((size_t)((long long)row.t0 * G / (NQ * KP_ROWS)) + r + (size_t)(base / (NQ * KP_ROWS))) * c.Hkv + h;
        float4* fold = reinterpret_cast<float4*>(p.ws + kp_part_floats(most, all_rows, HD)) +
                       (fold_tile * most + sp) * (NQ * KP_ROWS * HD / 4) + x * (KP_ROWS * HD / 4) + m;   // + KP_ROWS * (column / 4)
        float M_fold = -INFINITY;   // the maximum that the folded sums refer to
        auto fold_before = [&](int cc, float4 (&was)[16]) {   // columns cc .. cc + 63
            const bool some = live && M_fold != -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; ++e) was[e] = some ? fold[KP_ROWS * (cc / 4 + e)] : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        auto fold_o = [&](int cc, const float4 (&was)[16]) {
            const float f = M_fold == -INFINITY || M_fold == M ? 1.f : kv8_exp2(M_fold - M);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t o[32];
                tm_ld32(ocol + cc + 32 * q, o);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 w = was[8 * q + e];
                    if (live && M != -INFINITY)
                        fold[KP_ROWS * (cc / 4 + 8 * q + e)] =
                            make_float4(fmaf(w.x, f, __uint_as_float(o[4 * e])), fmaf(w.y, f, __uint_as_float(o[4 * e + 1])),
                                        fmaf(w.z, f, __uint_as_float(o[4 * e + 2])), fmaf(w.w, f, __uint_as_float(o[4 * e + 3])));
                }
            }
        };
        // Every phase of every barrier of the loop is waited for before the next can end, since a parity tells a phase only
        // from the one before it: s_full and p_full have a barrier for each S buffer, S of tile j + 2 follows P V of tile j,
        // and that P of tile j
        auto s_wait = [&](int j) { return warp_wait(&s_full[2 * x + (j & 1)], (uint32_t)(j >> 1) & 1u, ab, p.b.err); };
        // P V of tile j (asked at tile j + 1, or behind the last) is done: S of tile j + 2 follows it on the tensor core, and
        // does not wait for P of tile j + 1; the last two tiles have a barrier each
        auto pv_wait = [&](int j) {
            return j + 2 < ntiles ? s_wait(j + 2) : warp_wait(&pv_done[2 * x + (j == ntiles - 1)], 0u, ab, p.b.err);
        };
        for (int j = 0; j < (x < nact ? ntiles : 0); ++j) {
            const int k0 = key0(i0 + j);
            const bool folds = FINE && j > 0 && j % KP_FOLD == 0;
            if (folds) {   // the next P V starts O anew, after P of this tile is full
                float4 was[16];
                fold_before(0, was);   // on their way during the wait
                if (!(ok = pv_wait(j - 1))) break;
                fence_after();
#pragma unroll
                for (int cc = 0; cc < HD; cc += 64) {
                    if (cc) fold_before(cc, was);
                    fold_o(cc, was);
                }
                M_fold = M;
            }
            uint64_t* const mb = &meta_full[j % KP_META];
            const uint32_t mp = (uint32_t)(j / KP_META) & 1u;
            if (!__all_sync(0xffffffffu, mbar_try_wait(&s_full[2 * x + (j & 1)], (uint32_t)(j >> 1) & 1u) & mbar_try_wait(mb, mp)))
                ok = s_wait(j) && warp_wait(mb, mp, ab, p.b.err);
            if (!ok) break;
            fence_after();
            const uint32_t scol = lrow + 128 * x + 64 * (j & 1);
            const KpMeta* mt = meta[j % KP_META];
            uint32_t v[2][32];
            tm_ld32(scol, v[0]);
            tm_ld32(scol + 32, v[1]);
            wait_ld();
            // some row of the query tile does not see some of these positions
            if (!(xmin >= 0 && k0 + KP_KEYS - 1 <= xmin && (k0 > xmax - p.window || k0 + KP_KEYS - 1 < p.sinks))) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // bit e: position k0 + 32 q + e is one that this row sees
                    auto below = [&](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
                    const int kq = k0 + 32 * q;
                    const uint32_t see = below(pos + 1 - kq) & (~below(lo - kq) | below(p.sinks - kq));
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[q][e] = see >> e & 1u ? v[q][e] : 0xFF800000u;
                }
            }
            float mul[KP_GROUPS], add[KP_GROUPS], top = -INFINITY;
#pragma unroll
            for (int b = 0; b < KP_GROUPS; ++b) {
                auto f = [&](int e) { return __uint_as_float(v[b / 2][b % 2 * 16 + e]); };
                const float t0 = max3(f(0), f(1), f(2)), t1 = max3(f(3), f(4), f(5)), t2 = max3(f(6), f(7), f(8));
                const float t3 = max3(f(9), f(10), f(11)), t4 = max3(f(12), f(13), f(14));
                const float2 k = *reinterpret_cast<const float2*>(&mt[b]);
                mul[b] = kp_mul(fac, k.x);
                add[b] = k.y;
                top = fmaxf(top, fmaf(fmaxf(max3(t0, t1, t2), max3(t3, t4, f(15))), mul[b], add[b]));
            }
            float alpha = 1.f;
            if (top > M + KP_SLACK) {
                if (M != -INFINITY) alpha = kv8_exp2(M - top);   // else nothing has been summed yet
                M = top;
                l *= alpha;
            }
            bool waited = j == 0 || folds;   // for P V of tile j - 1
            if (!waited && __any_sync(0xffffffffu, alpha != 1.f)) {
                if (!(ok = pv_wait(j - 1))) break;
                waited = true;
                fence_after();
#pragma unroll 1
                for (int cc = 0; cc < HD; cc += 16) {
                    uint32_t o[16];
                    tm_ld16(ocol + cc, o);
                    wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tm_st16(ocol + cc, o);
                }
            }
            const float sub = (M == -INFINITY ? 0.f : M) - KP_SHIFT;
            const uint64_t minus2 = pair(-1.f, -1.f), less2 = pair(-sub, -sub);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t hi[16], low[16], third[FINE ? 16 : 1];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float mu = mul[2 * q + b], plus = add[2 * q + b];
                    const uint64_t by = pair(mu, mu), plus2 = pair(plus, plus);
                    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float w0, w1;
                        // rounded before M is subtracted: M is a rounded score, and past 2^24 an unrounded one may lie far from
                        // it.  (mul.f32x2 and add.f32x2 would be fused by the assembler; a sum with what it does not know is not)
                        unpair(add2(fma2(pair(__uint_as_float(v[q][16 * b + e]), __uint_as_float(v[q][16 * b + e + 1])), by, plus2), less2), w0, w1);
                        w0 = kv8_exp2(w0);
                        w1 = kv8_exp2(w1);
                        if (e == 0) sum0 = pair(w0, w1);
                        else if (e == 2) sum1 = pair(w0, w1);
                        else if (e & 2) sum1 = add2(sum1, pair(w0, w1));
                        else sum0 = add2(sum0, pair(w0, w1));
                        const int d = 8 * b + e / 2;
                        hi[d] = pack_b2(w0, w1);
                        float r0, r1;
                        unpair(fma2(pair(__uint_as_float(hi[d] << 16), __uint_as_float(hi[d] & 0xFFFF0000u)), minus2, pair(w0, w1)), r0, r1);
                        low[d] = pack_b2(r0, r1);
                        if constexpr (FINE) {
                            unpair(fma2(pair(__uint_as_float(low[d] << 16), __uint_as_float(low[d] & 0xFFFF0000u)), minus2, pair(r0, r1)), r0, r1);
                            third[d] = pack_b2(r0, r1);
                        }
                    }
                    float a0, a1;
                    unpair(add2(sum0, sum1), a0, a1);
                    l += a0 + a1;
                }
                tm_st16(scol + 16 * q, hi);   // over the scores, which this thread holds
                tm_st16(scol + 32 + 16 * q, low);
                if constexpr (LY::THIRD_TMEM) tm_st16(lrow + LY::THIRD + 64 * x + 32 * (j & 1) + 16 * q, third);
                if constexpr (LY::THIRD_SMEM) {
                    if (q == 0 && !waited && !(ok = pv_wait(j - 1))) break;   // that read the third parts of its tile
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(sm + LY::P3 + x * LY::PTILE + kp_sw(m, 4 * q + e)) =
                            make_uint4(third[4 * e], third[4 * e + 1], third[4 * e + 2], third[4 * e + 3]);
                }
            }
            if (!ok) break;
            if constexpr (LY::THIRD_SMEM) fence_proxy_async_smem();
            wait_st();
            fence_before();
            mbar_arrive(&p_full[2 * x + (j & 1)]);
        }
        if (x < nact && ok && ntiles > 0) {
            ok = pv_wait(ntiles - 1);
            fence_after();
        }
        cta_meet();   // every tile has been converted: the marks are complete
        if (x < nact && ok) {
            // NaN in V that this row sees: a bit for each column
            uint32_t nan[HD / 32];
#pragma unroll
            for (int d = 0; d < HD / 32; ++d) nan[d] = 0u;
            if (marked) {
                for (int j = i0; j < i1; ++j) {
                    if (!(marks[j / 32 % KP_MARKS] >> (j & 31) & 1u)) continue;
                    const int k0 = key0(j);
                    for (int key = k0; key < min(k0 + KP_KEYS, pos + 1); ++key) {
                        if (!kv8_sees(pos, key, p.window, p.sinks)) continue;
                        const int id = c.pages ? c.pages[(size_t)r * c.ppr + key / c.page] : r * c.ppr + key / c.page;
                        if ((unsigned)id >= (unsigned)c.num_pages) continue;
                        const uint32_t* w = reinterpret_cast<const uint32_t*>(
                            c.v + (((size_t)id * c.Hkv + h) * c.page + key % c.page) * HD);
#pragma unroll
                        for (int d = 0; d < HD / 32; ++d)
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t n = nan_bytes(__ldg(w + 8 * d + e)) >> 7;   // bits 0, 8, 16, 24
                                nan[d] |= ((n & 1u) | (n >> 7 & 2u) | (n >> 14 & 4u) | (n >> 21 & 8u)) << (4 * e);
                            }
                    }
                }
            }
            // Each thread has a row; memory wants rows side by side.  So a warp lays its 32 rows down in shared memory,
            // which nobody needs any more (16-byte chunks permuted against bank conflicts), and writes them row by row:
            // 16 bytes of 32 rows at a time cost some 2 us a CTA
            const bool whole = splits == 1;
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const int bytes = whole ? HD * (int)sizeof(T) : HD * 4, log2_chunks = 31 - __clz(bytes / 16);   // 8, 16 or 32 a row
            unsigned char* stage = sm + warp * (32 * HD * 4);
#pragma unroll
            for (int cc = 0; cc < HD; cc += 16) {
                uint32_t o[16];
                if (ntiles > 0) {
                    tm_ld16(ocol + cc, o);
                    wait_ld();
                    if (FINE && live && M_fold != -INFINITY) {   // and what is folded
                        const float f = kv8_exp2(M_fold - M);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 w = fold[KP_ROWS * (cc / 4 + e)];
                            o[4 * e] = __float_as_uint(fmaf(w.x, f, __uint_as_float(o[4 * e])));
                            o[4 * e + 1] = __float_as_uint(fmaf(w.y, f, __uint_as_float(o[4 * e + 1])));
                            o[4 * e + 2] = __float_as_uint(fmaf(w.z, f, __uint_as_float(o[4 * e + 2])));
                            o[4 * e + 3] = __float_as_uint(fmaf(w.w, f, __uint_as_float(o[4 * e + 3])));
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (nan[cc / 32] >> (cc % 32 + e) & 1u) o[e] = 0x7FFFFFFFu;
                    o[e] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);   // nothing seen: O is undefined
                }
                auto lay = [&](int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
                    *reinterpret_cast<uint4*>(stage + lane * bytes + ((chunk ^ (lane & 7)) << 4)) = make_uint4(x, y, z, w);
                };
                if (FINE || !whole) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) lay((cc + e) / 4, o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else {
                    auto two = [&](int e) { return pack_bf16x2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])); };
#pragma unroll
                    for (int e = 0; e < 16; e += 8) lay((cc + e) / 8, two(e), two(e + 2), two(e + 4), two(e + 6));
                }
            }
            __syncwarp();
            const unsigned long long to = live ? (unsigned long long)(whole ? (void*)dst : (void*)piece) : 0ull;
            for (int k = 0; k < 1 << log2_chunks; ++k) {
                const int i = k * 32 + lane, rr = i >> log2_chunks, chunk = i & ((1 << log2_chunks) - 1);
                const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * bytes + ((chunk ^ (rr & 7)) << 4));
                const unsigned long long at = __shfl_sync(0xffffffffu, to, rr);
                if (at) reinterpret_cast<uint4*>(at)[chunk] = v;
            }
            if (splits > 1 && live) {
                float* ml = p.ws + (size_t)most * all_rows * HD + (sp * all_rows + qrow) * 2;
                ml[0] = M;
                ml[1] = l;
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == KP_MMA_WARP) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(dt) : "memory");
    }
}

// one warp for each token and query head: the splits' parts in split order.  grid (query rows / 8, rows)
template <int HD, bool FINE>
__global__ void __launch_bounds__(256) k_kv8_prompt_join(const Kv8Attend p, int most) {
    using T = typename std::conditional<FINE, float, __nv_bfloat16>::type;
    pdl_wait();
    const int r = blockIdx.y, lane = threadIdx.x & 31;
    const long long m = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    Kv8Row row;
    if (!kv8_row(p.b, p.c.ppr * p.c.page, r, &row) || m >= (long long)row.n * p.Hq) return;
    // the parts of the CTA that had this query row
    const int tk = (int)(m / p.Hq), g = (int)(m % p.Hq) % p.G, base = (tk * p.G + g) / (2 * KP_ROWS) * (2 * KP_ROWS), p0 = row.len - row.n;
    const KpTiles tl = kp_tiles(p0 + p.by_group.of(base), p0 + p.by_group.of(min(base + 2 * KP_ROWS, row.n * p.G) - 1), p.window, p.sinks);
    const int splits = kp_parts(tl.n, most);
    if (splits == 1) return;   // it wrote the result itself
    const size_t all_rows = (size_t)p.b.total * p.Hq, qrow = (size_t)row.t0 * p.Hq + m;
    const float* ml = p.ws + (size_t)most * all_rows * HD;
    constexpr int D = HD / 32;
    // lane s knows of part s: its maximum, sum and weight.  A part that saw nothing is all zeros with weight 0
    const float2 mine = lane < splits ? *reinterpret_cast<const float2*>(ml + (lane * all_rows + qrow) * 2) : make_float2(-INFINITY, 0.f);
    const float M = warp_max(mine.x), weight = mine.x == -INFINITY ? 0.f : kv8_exp2(mine.x - M);
    float l = 0.f, o[D];
#pragma unroll
    for (int d = 0; d < D; ++d) o[d] = 0.f;
    const float* part = p.ws + qrow * HD + lane * D;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {   // the parts' loads do not wait for one another
        const float f = __shfl_sync(0xffffffffu, weight, s);
        l = fmaf(__shfl_sync(0xffffffffu, mine.y, s), f, l);
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = fmaf(part[s * all_rows * HD + d], f, o[d]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* dst = static_cast<T*>(p.out) + (row.t0 + m / p.Hq) * p.out_stride + m % p.Hq * HD + lane * D;
#pragma unroll
    for (int d = 0; d < D; ++d) Elem<T>::round_store(o[d] * inv, dst + d);
}

long long prompt_tiles(const Kv8Attend& p) {   // query tiles (of one CTA) of the longest row
    const int per = 2 * KP_ROWS;
    return ((long long)p.b.max_new * p.G + per - 1) / per;
}

long long prompt_keys(const Kv8Attend& p) {   // the most positions that the rows of a CTA may see, and two tiles
    const long long keys = (long long)p.c.ppr * p.c.page, win = (long long)p.window + p.sinks + p.b.max_new;
    return (win < keys ? win : keys) + 2 * KP_KEYS;
}
// The most parts: as many as bring the CTAs to one round of the SMs (a second round costs more than it saves: a prompt
// of 1024 tokens, 128 CTAs of up to 16 tiles, takes 31 us whole and 50 us in parts of 8)
int prompt_splits(const Kv8Attend& p, int num_sms) {
    const long long ctas = prompt_tiles(p) * p.c.Hkv * p.c.rows, tiles = prompt_keys(p) / KP_KEYS;
    long long n = num_sms / ctas;
    if (n > 32) n = 32;   // the join's lanes
    return n < 1 ? 1 : kp_parts((int)(tiles < (1 << 20) ? tiles : 1 << 20), (int)n);
}

template <int HD, bool FINE>
cudaError_t launch(const Kv8Attend& p, int num_sms, cudaStream_t s) {
    const int splits = prompt_splits(p, num_sms);
    static OncePerDevice raised;
    cudaError_t e = raised.run([] {
        return cudaFuncSetAttribute((const void*)&k_kv8_prompt<HD, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kp_smem<HD, FINE>());
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(prompt_tiles(p) * p.c.Hkv), p.c.rows * splits);
    cfg.blockDim = dim3(KP_THREADS);
    cfg.dynamicSmemBytes = kp_smem<HD, FINE>();
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_kv8_prompt<HD, FINE>, p, splits);
    if (e != cudaSuccess || splits == 1) return e;
    cfg.gridDim = dim3((unsigned)(((long long)p.b.max_new * p.Hq + 7) / 8), p.c.rows);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_kv8_prompt_join<HD, FINE>, p, splits);
}

}  // namespace

size_t kv8_prompt_floats(const Kv8Attend& p, int num_sms) {
    const int splits = prompt_splits(p, num_sms);
    size_t n = kp_part_floats(splits, (size_t)p.b.total * p.Hq, p.c.hd);
    // fp32 q and more tiles than O takes unfolded: a fold for each query tile of each row
    // (a part holds at most 8 tiles, or its share of all of them)
    const long long tiles_most = prompt_keys(p) / KP_KEYS + 2;
    if (p.dtype == W_F32 && (tiles_most + splits - 1) / splits + 1 > KP_FOLD) {
        const size_t tiles = (size_t)p.b.total * p.G / (2 * KP_ROWS) + p.c.rows + 1;
        n += tiles * p.c.Hkv * splits * (2 * KP_ROWS) * p.c.hd;
    }
    return n;
}

cudaError_t kv8_prompt_launch(const Kv8Attend& p, int num_sms, cudaStream_t s) {
    const bool fine = p.dtype == W_F32;
    if (p.c.hd == 128) return fine ? launch<128, true>(p, num_sms, s) : launch<128, false>(p, num_sms, s);
    return fine ? launch<64, true>(p, num_sms, s) : launch<64, false>(p, num_sms, s);
}

}  // namespace gd
