// kv8_decode.cu -- attention over the 8-bit K/V cache for single tokens (and for
// the few tokens of a draft): up to 16 query rows a launch (tokens x the query heads of a
// K/V head) against one K/V head of one sequence.
//
// Bound: the bytes of the visible K and V, each read once.  Everything else has
// to hide behind that stream, so
//   * each warp copies its own 16-key steps into a ring in shared memory (cp.async,
//     three steps ahead, seven at 64 dims), so most of an SM's shared memory is
//     in flight, whatever registers the arithmetic needs.  No barrier joins the
//     warps inside the loop;
//   * both products keep the cache as the A operand of mma.m16n8k16
//     (S^T = K Q^T, O^T = V^T P^T), so the few query rows fill the N = 8 side and
//     no accumulator row is wasted.  The sum over dims may run in any order: lane
//     (g, t) of a warp takes consecutive bytes of key g as its operand words, q is
//     laid out to match; for V a lane takes a run of dims of its four keys and
//     pairs the keys' bytes with byte permutes.  No transposing load; 16-byte
//     chunks are permuted within the rows so that both reads are free of bank
//     conflicts;
//   * e4m3 converts to f16 exactly and in pairs; the scales stay outside the
//     products: K's exponent multiplies the 16-key score tile, V's the step's
//     P V where it is added to the result in fp32;
//   * q enters as two f16 parts (22 bits; exact for bf16, whose second part is
//     not multiplied), the weights as two f16 parts for either type;
//   * the maximum is kept within a factor 4 of the true one (weights are scaled
//     by 2^13, f16 holds 2^15), so a 16-key step needs one vote and almost never
//     a reduction or a rescaling;
//   * two f16 parts hold only some 27 bits below the largest weight, and the
//     largest may belong to a position whose V is 0 in a dim.  The same vote finds
//     a step with smaller weights.  It is taken relative to its own largest, and
//     where its 16 weights lie further apart than that, it is marked, and computed
//     again for the rest when the loop is done;
//   * work: the visible 16-key steps of each row and K/V head (windows make gaps
//     that are never touched).  Where the places (two CTAs an SM) suffice, each
//     (row, head) is cut into pieces of its own, of at least two steps a warp, so
//     short rows are not cut.  Otherwise all steps, in one line, are cut into
//     equal pieces, one for each place, whatever the lengths are.  A (row, head)
//     that is cut leaves partial results in the workspace; the CTA that finishes
//     it last joins them, in the order of the pieces, and sets its counter back
//     to 0: one launch.
//
// Measured (128 dims): 32 bf16 rows of up to 32k positions 227 us, 6.2 TB/s or
// 92 % of the measured copy rate (222 with weights of one f16 part and nothing for
// the small ones; with queries twice and four times as long, whose scores lie
// further apart, 256 and 477); 8 fp32 rows x 8k 30.8 us and one row of 8191
// 13.9 us, where the ends bind it: of the 7.4 us that one short row takes on the
// device, the launch, the plan (a trip to the lengths), the first steps (page id,
// then bytes) and the join's trip through memory are nearly all.  Two CTAs an SM
// hide one's ends behind the other's stream: when it was changed, a single CTA of
// 12 warps took 34.6 us for the 8 rows, three of 4 warps 31.
#include <limits.h>
#include <type_traits>
#include "kv8.cuh"
#include "mma_helpers.cuh"

namespace gd {

namespace {

constexpr int KD_STEP = 16;           // positions of a step: the unit of work
constexpr float KD_SLACK = 1.f;       // how far the maximum, rounded down, may lag (log2)
constexpr float KD_SHIFT = 13.f;      // weights carry 2^13: M is the maximum less 13
constexpr float KD_NONE = -3.402823466e38f;   // M before the first score: any is above it by more than the slack
// Two f16 parts hold a weight of 2^(x - KD_SHIFT) of M's to 11 bits from x = -14 on; where the second carries KD_LOW, as
// with fp32 q, to 20 bits from x = -17 on: KD_DEEP below the largest.  A step with smaller weights is taken relative to
// its own largest, which gets another bit, and what lies more than KD_SPAN below that waits for a pass of its own.
// Weights below 2^-KD_LAST of the largest are 0 in fp32.  (The hundredth: no rounding lets a step that is not taken
// relative to its own largest hold a weight below KD_SPAN.)
template <bool FINE>
constexpr int KD_SPAN = FINE ? 31 : 28;
template <bool FINE>
constexpr float KD_DEEP = KD_SPAN<FINE> - 1.01f;
constexpr float KD_LOW = 0x1p12f, KD_LAST = 126.f;
constexpr float KD_UNIT = 0x1p-14f;   // results are summed in this unit, so that no term is above V's own size

// a row of which only the tokens [skip, skip + take) count: it ends behind them
__device__ __forceinline__ Kv8Row kd_some(const Kv8Row& row, int skip, int take) {
    const int n = min(max(row.n - skip, 0), take);
    return Kv8Row{row.t0 + skip, n, max(row.len - max(row.n - skip - n, 0), 0)};
}

// The steps of a row: its first `sink` steps, then `gap` that no token sees,
// then the rest; n of them are visible to one of its tokens.
struct KdSteps {
    int n, sink, gap;
};
__device__ __forceinline__ KdSteps kd_steps(const Kv8Row& row, int window, int sinks) {
    if (row.n == 0) return KdSteps{0, 0, 0};
    const int end = (row.len + KD_STEP - 1) / KD_STEP;
    const int first = max(row.len - row.n, 0);
    const int low = (int)max((long long)first - window + 1, 0ll) / KD_STEP;   // the first token's window begins here
    const int sink = (min(sinks, row.len) + KD_STEP - 1) / KD_STEP;
    if (sink >= low) return KdSteps{max(end, 1), end, 0};   // a row without positions has one step with nothing in it
    return KdSteps{sink + end - low, sink, low - sink};
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// a / b for a >= 0: most numbers here fit 32 bits, and a 64-bit division costs a short call half a microsecond
__device__ __noinline__ long long quotient64(long long a, int b) { return a / b; }
__device__ __forceinline__ long long quotient(long long a, int b) {
    return (a >> 32) ? quotient64(a, b) : (long long)((uint32_t)a / (uint32_t)b);
}
// The work cut into pieces.  own: pieces of one (row, head) each; else the line of units in pieces of q or q + 1
struct KdCut {
    bool own;
    int pieces, rem;
    long long units, q;
    __device__ __forceinline__ long long begin(int c) const { return q * c + min(c, rem); }
    __device__ __forceinline__ int piece_of(long long u) const {
        const long long lead = (q + 1) * rem;   // q < 2^31: a piece is a part of one SM's work
        return u < lead ? (int)quotient(u, (int)q + 1) : rem + (int)quotient(u - lead, (int)q);
    }
};
// The plan is made by every warp for itself, 32 rows at a time and a row for each lane: no shared memory, no
// barrier, and one trip to memory where there are at most 32 rows
struct KdRows {
    const Kv8Attend& p;
    const int lane, cap;
    int at = -1, n = 0;   // the 32 rows held: 32 * at .., steps of row 32 * at + lane
    Kv8Row row{0, 0, 0};  // and what it is
    __device__ __forceinline__ KdRows(const Kv8Attend& p_) : p(p_), lane(threadIdx.x & 31), cap(p_.c.ppr * p_.c.page) {}
    __device__ __forceinline__ int steps(int chunk) {
        if (chunk != at) {
            const int r = 32 * chunk + lane;
            n = 0;
            if (r < p.c.rows && kv8_row(p.b, cap, r, &row)) {
                if (p.take) row = kd_some(row, p.skip, p.take);
                n = kd_steps(row, p.window, p.sinks).n;
            }
            at = chunk;
        }
        return n;
    }
    __device__ __forceinline__ int chunks() const { return (p.c.rows + 31) / 32; }
};
// a row's pieces: least > 0: cuts of at least that many steps; 0: its steps
__device__ __forceinline__ uint32_t kd_weight(int n, int least) { return least ? (uint32_t)((n + least - 1) / least) : (uint32_t)n; }
// Row and place of item u on the line of all heads' weights: the weight of the rows before (of one head) and of the row
struct KdPlace {
    int r;
    Kv8Row row;
    long long before;
    uint32_t weight;
};
__device__ __forceinline__ KdPlace kd_find(KdRows& rows, long long u, int least) {
    const int Hkv = rows.p.c.Hkv;
    long long before = 0;
    for (int k = 0; k < rows.chunks(); ++k) {
        const uint32_t w = kd_weight(rows.steps(k), least);
        uint32_t inc = w;   // 32 rows of at most 2^26 steps
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (rows.lane >= o) inc += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, (before + inc) * Hkv > u);
        if (past) {   // the first row that ends behind u
            const int l = __ffs(past) - 1;
            const uint32_t wl = __shfl_sync(0xffffffffu, w, l);
            const Kv8Row row{__shfl_sync(0xffffffffu, rows.row.t0, l), __shfl_sync(0xffffffffu, rows.row.n, l),
                             __shfl_sync(0xffffffffu, rows.row.len, l)};
            return KdPlace{32 * k + l, row, before + __shfl_sync(0xffffffffu, inc, l) - wl, wl};
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return KdPlace{-1, Kv8Row{0, 0, 0}, 0, 0};   // the lengths have changed under the kernel: nothing is left to do
}
template <int W>
__device__ __forceinline__ KdCut kd_plan(KdRows& rows, int grid, int* least) {
    const int Hkv = rows.p.c.Hkv;
    long long all = 0, all_cuts = 0;
    for (int k = 0; k < rows.chunks(); ++k) all += __reduce_add_sync(0xffffffffu, (uint32_t)rows.steps(k));
    KdCut cut;
    cut.units = all * Hkv;
    // Own pieces: the places that stay without work cost more the longer the pieces are, a piece that goes on in a
    // second head costs some 4 us.  So an eighth may idle up to 512 steps a place, three up to 96, none beyond
    // (16 rows x 4 heads x 257 steps: 22.9 us with own pieces, 26.2 without; 32 x 8 x ~1350: 306 against 221)
    all_cuts = grid + 1;
    for (int spare = 9; spare <= 11 && all_cuts * Hkv > grid; spare += 2) {
        if (cut.units > (spare == 9 ? 512ll : 96ll) * grid) break;
        *least = (int)max(2ll * W, quotient(cut.units * spare + 8 * grid - 1, 8 * grid));
        all_cuts = 0;
        for (int k = 0; k < rows.chunks(); ++k) all_cuts += __reduce_add_sync(0xffffffffu, kd_weight(rows.steps(k), *least));
    }
    cut.own = all_cuts * Hkv <= grid;
    cut.pieces = cut.own ? (int)all_cuts * Hkv : grid;
    cut.q = quotient(cut.units, grid);   // at least 1 where it is used: more units than pieces
    cut.rem = (int)(cut.units - cut.q * grid);
    return cut;
}
template <int HD, int MT>
__host__ __device__ constexpr int kd_slot_floats() { return MT * 8 * (HD + 2); }   // O, then M, then l of each query row

// A step is 16 positions: K, then V, 16 rows of HD bytes each in lines of 128.
// Chunk x (16 bytes) of row `key` lies at kd_at: chunks are permuted so that the
// rows that a quarter warp reads at once lie in different banks.
template <int HD>
__device__ __forceinline__ uint32_t kd_at(int key, int x) {
    if constexpr (HD == 128) return (uint32_t)(key * 128 + ((x ^ (key & 7)) << 4));
    else return (uint32_t)((key >> 1) * 128 + (((((key & 1) << 2) | x) ^ ((key & 6))) << 4));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// dynamic shared memory: the rings; when the loop is done the warps' results lie over them
template <int HD, int MT>
struct KdShared {
    static constexpr int W = MT == 1 ? 6 : 4, CTAS = 2;   // warps of a CTA, CTAs on an SM: one's ends hide behind the other's stream
    static constexpr int STEP = 2 * KD_STEP * HD, STAGES = 512 / HD;   // 16 KB a warp
    static constexpr int RING = W * STAGES * STEP, OUT = W * MT * 8 * HD * (int)sizeof(float);
    static constexpr int BYTES = RING > OUT ? RING : OUT;
};

// MT: query rows / 8 (up).  FINE: fp32 q -- second f16 parts of q and of the weights.
template <int HD, int MT, bool FINE>
__global__ void __launch_bounds__(32 * KdShared<HD, MT>::W, KdShared<HD, MT>::CTAS) k_kv8_decode(const Kv8Attend p) {
    using T = typename std::conditional<FINE, float, __nv_bfloat16>::type;
    constexpr int NK = HD / 16;   // 16-dim steps of S, 16-dim tiles of O
    constexpr int PARTS = FINE ? 2 : 1, STAGES = KdShared<HD, MT>::STAGES, W = KdShared<HD, MT>::W;
    extern __shared__ __align__(128) unsigned char kd_raw[];
    float(*o_s)[MT * 8][HD] = reinterpret_cast<float(*)[MT * 8][HD]>(kd_raw);
    const unsigned char* ring_p = kd_raw + (threadIdx.x >> 5) * (STAGES * KdShared<HD, MT>::STEP);
    const uint32_t ring = smem_u32(ring_p);
    __shared__ int last_s;
    __shared__ float m_s[W][MT * 8], l_s[W][MT * 8];
    __shared__ __align__(16) uint4 q_s[PARTS][MT][NK / 2][32];   // f16 parts of q, by step and lane
    __shared__ float fac_s[MT * 8];
    __shared__ uint32_t nan_s[W][HD];
    pdl_wait();
    const Kv8Cache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = p.G, nb = c.page >> c.block_log2;
    KdRows rows(p);
    int least = 1;
    const KdCut cut = kd_plan<W>(rows, gridDim.x, &least);
    if ((int)blockIdx.x >= cut.pieces) return;
    const long long u_begin = cut.own ? blockIdx.x : cut.begin(blockIdx.x);
    const long long u_end = cut.own ? u_begin + 1 : cut.begin(blockIdx.x + 1);

    for (long long u = u_begin; u < u_end;) {
        // steps [i0, i1) of row r and K/V head h; a head that is cut has the pieces c0 .. c1
        const KdPlace at = kd_find(rows, u, cut.own ? least : 0);
        const int r = at.r;
        if (r < 0) break;
        const Kv8Row row = at.row;
        const KdSteps tl = kd_steps(row, p.window, p.sinks);
        const long long in_row = u - at.before * c.Hkv;
        const int h = (int)quotient(in_row, (int)at.weight), in_head = (int)(in_row - (long long)h * at.weight);
        int i0, i1, c0, c1;
        if (cut.own) {
            c0 = blockIdx.x - in_head;
            c1 = c0 + (int)at.weight - 1;
            i0 = (int)quotient((long long)tl.n * in_head, (int)at.weight);
            i1 = (int)quotient((long long)tl.n * (in_head + 1), (int)at.weight);
        } else {
            i0 = in_head;
            i1 = (int)min((long long)tl.n, i0 + (u_end - u));
            c0 = cut.piece_of(u - i0);
            c1 = cut.piece_of(u - i0 + tl.n - 1);
        }
        const int nq = row.n * G, p0 = row.len - row.n;   // query rows, the first token's position

        const int end = min(row.len, p0 + row.n);
        const int low = (int)max((long long)max(p0, 0) - p.window + 1, 0ll);   // no token of the row sees [sinks, low)
        // this warp's steps: i0 + warp + k * W, k < mine
        const int mine = max((i1 - i0 - warp + W - 1) / W, 0);
        auto key0 = [&](int k) {
            const int i = i0 + warp + k * W;
            return (i < tl.sink ? i : i + tl.gap) * KD_STEP;
        };
        auto wanted = [&](int kb) { return kb < end && (kb + 15 >= low || kb < p.sinks); };
        // 32 of them, one for each lane: where in the pools, in 16 rows (-1: no step), and the scale bytes.  The copies
        // run ahead of the arithmetic: it may still need the 32 before.
        int place = -1, place_before = -1, ke = 0, ke_before = 0, ve = 0, ve_before = 0;
        auto check_scales = [&]() {   // of the 32 held, once they are here: a check in every step takes 3 % of the time
            if (place >= 0 && !(kv8_scale_ok(ke) && kv8_scale_ok(ve))) atomicOr(p.b.err, FAULT_SCALE);
        };
        auto next32 = [&](int k) {
            check_scales();
            place_before = place;
            ke_before = ke;
            ve_before = ve;
            place = -1;
            if (k + lane >= mine) return;
            const int kb = key0(k + lane);
            if (!wanted(kb)) return;
            const int slot = c.by_page.of(kb), off = kb - slot * c.page, page = kv8_page(c, p.b.err, r, slot);
            if (page < 0) return;
            const long long head = (long long)page * c.Hkv + h;
            place = (int)((head * c.page + off) >> 4);
            const long long at = head * nb + (off >> c.block_log2);
            ke = c.ks[at];   // not looked at before the step is computed: nothing waits for them here
            ve = c.vs[at];
        };
        // the step of lane l of the 32 into a stage of the ring
        auto copy_step = [&](int l, int stage) {
            const int there = __shfl_sync(0xffffffffu, place, l);
            if (there < 0) return;
            const size_t at = (size_t)there * (16 * HD);
            const uint32_t dst = ring + (uint32_t)(stage * KdShared<HD, MT>::STEP);
#pragma unroll
            for (int u = 0; u < HD / 32; ++u) {
                const int x = lane + 32 * u;
                const uint32_t d = dst + kd_at<HD>(x / (HD / 16), x % (HD / 16));
                copy16(d, c.k + at + (size_t)x * 16);
                copy16(d + 16 * HD, c.v + at + (size_t)x * 16);
            }
        };
        int ahead = 0;   // the next step to copy
        // one more step into the ring; one group a call, also for nothing
        auto copy_next = [&]() {
            const int i = ahead++;
            if (i < mine) {
                if ((i & 31) == 0) next32(i);
                copy_step(i & 31, i % STAGES);
            }
            copy_commit();
        };
        // q on its way before the first page id is waited for.  The sets of 8 query rows and the pairs of 16 dims are laid
        // out by different warps; each needs all of a row for its power of two
        constexpr int QW = HD / 4 / Elem<T>::VEC;   // 16-byte words of a lane's dims
        constexpr int PAIRS = NK / 2, ITEMS = MT * PAIRS;
        auto load_q = [&](int a, uint4 (&qw)[QW]) {
            const int m = a * 8 + g;
            const int n = p.by_group.of(m);
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (row.t0 + n) * p.q_stride +
                                                              (h * G + m - n * G) * HD + t * (HD / 4));
#pragma unroll
            for (int v = 0; v < QW; ++v) qw[v] = m < nq ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 qw[QW];
        if (warp < ITEMS) load_q(warp / PAIRS, qw);
#pragma unroll
        for (int x = 0; x < STAGES - 1; ++x) copy_next();   // in flight while q is laid out

        // q as B operand: lane (g, t) holds 16 dims' worth of query row g of a set
        float fac[MT][2];   // scale * log2(e) / q's power of two, of query rows 2t and 2t + 1
        int pos[MT][2];     // their positions (-1: no such row, or before the sequence)
        for (int item = warp; item < ITEMS; item += W) {
            const int a = item / PAIRS, pr = item % PAIRS;
            if (item != warp) load_q(a, qw);
            float top = 0.f, mine4[8];   // this pair's 8 values of the lane
#pragma unroll
            for (int v = 0; v < QW; ++v) {
                float f[Elem<T>::VEC];
                Elem<T>::unpack(qw[v], f);
#pragma unroll
                for (int e = 0; e < Elem<T>::VEC; ++e) {
                    top = fmaxf(top, fabsf(f[e]));
                    if ((v * Elem<T>::VEC + e) / 8 == pr) mine4[(v * Elem<T>::VEC + e) % 8] = f[e];
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // a power of two that brings the row's largest value to [2^14, 2^15)
            const int ex = min(max(268 - (int)(__float_as_uint(top) >> 23), 1), 254);
            const float up = __int_as_float(ex << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float x0 = mine4[2 * b] * up, x1 = mine4[2 * b + 1] * up;
                hi[b] = pack_f16x2(x0, x1);
                const float2 f = unpack_f16x2(hi[b]);
                lo[b] = pack_f16x2(x0 - f.x, x1 - f.y);
            }
            q_s[0][a][pr][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (FINE) q_s[1][a][pr][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (pr == 0 && t == 0) fac_s[a * 8 + g] = p.scale * KV8_LOG2E / up;
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int mq = a * 8 + 2 * t + b;
                fac[a][b] = fac_s[mq];
                pos[a][b] = mq < nq ? p0 + p.by_group.of(mq) : -1;
            }

        float o[MT][NK][4], M[MT][2], l[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[a][k][e] = 0.f;
            M[a][0] = M[a][1] = KD_NONE;
            l[a][0] = l[a][1] = 0.f;
        }

        auto compute = [&](auto is_first, int i, int stage, int e_k, int e_v, int level) -> bool {
            constexpr bool FIRST = decltype(is_first)::value;
            const int kb = key0(i);
            const unsigned char* step = ring_p + stage * KdShared<HD, MT>::STEP;
            // S^T: rows keys g, g + 8; columns query rows 2t, 2t + 1
            float sc[MT][4], s1[MT][4];   // two chains of products are half as long as one
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[a][e] = s1[a][e] = 0.f;
#pragma unroll
            for (int j = 0; j < HD / 64; ++j) {
                const uint4 k0 = *reinterpret_cast<const uint4*>(step + kd_at<HD>(g, t * (HD / 64) + j));
                const uint4 k1 = *reinterpret_cast<const uint4*>(step + kd_at<HD>(g + 8, t * (HD / 64) + j));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
                    e4m3x4_to_f16(w0[e], a0, a2);
                    e4m3x4_to_f16(w1[e], a1, a3);
                    e4m3x4_to_f16(w0[e + 1], c0, c2);
                    e4m3x4_to_f16(w1[e + 1], c1, c3);
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int f = 0; f < PARTS; ++f) {
                            const uint4 q = q_s[f][a][(j * 4 + e) / 2][lane];
                            mma_f16(sc[a], a0, a1, a2, a3, q.x, q.y);
                            mma_f16(s1[a], c0, c1, c2, c3, q.z, q.w);
                        }
                }
            }
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[a][e] = __fadd_rn(sc[a][e], s1[a][e]);
            const float kf = pow2i(e_k);
            // positions every token of the row sees need no mask
            const bool all = kb + 15 <= p0 && (kb + 15 < p.sinks || kb > row.len - 1 - p.window);
            float by[MT][2], x[MT][4];   // x: log2 of the weights
            auto weigh = [&]() {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int b = e & 1, j = kb + g + (e >> 1) * 8;
                        x[a][e] = __fadd_rn(__fmul_rn(sc[a][e], by[a][b]), -M[a][b]);   // not fused: M is of rounded scores
                        if (!all && !(pos[a][b] >= 0 && kv8_sees(pos[a][b], j, p.window, p.sinks))) x[a][e] = -INFINITY;
                    }
            };
            float high = -INFINITY, low = INFINITY;
#pragma unroll
            for (int a = 0; a < MT; ++a) by[a][0] = __fmul_rn(fac[a][0], kf), by[a][1] = __fmul_rn(fac[a][1], kf);
            weigh();
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) high = fmaxf(high, x[a][e]), low = fminf(low, x[a][e]);
            float w[MT][4], unit[MT][2];   // weights, and what the product with them is worth for each query row
            bool deep = !FIRST, rest = false;
            if (FIRST && __any_sync(0xffffffffu, high > KD_SHIFT + KD_SLACK || low < KD_SHIFT - KD_DEEP<FINE>)) {
                if (__any_sync(0xffffffffu, high > KD_SHIFT + KD_SLACK)) {
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            float m = -INFINITY;
#pragma unroll
                            for (int e = b; e < 4; e += 2)
                                if (x[a][e] > -INFINITY) m = fmaxf(m, __fmul_rn(sc[a][e], by[a][b]));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                            m = fmaxf(__fadd_ru(floorf(m), -KD_SHIFT), M[a][b]);   // up: no weight above f16, whatever the scores
                            const float f = kv8_exp2(M[a][b] - m);
                            M[a][b] = m;
                            l[a][b] *= f;
#pragma unroll
                            for (int k = 0; k < NK; ++k) {
                                o[a][k][b] *= f;
                                o[a][k][b + 2] *= f;
                            }
                        }
                    weigh();
                }
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int e = 0; e < 4; ++e) deep |= x[a][e] < KD_SHIFT - KD_DEEP<FINE> && x[a][e] > KD_SHIFT - KD_LAST;
                deep = __any_sync(0xffffffffu, deep);
            }
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[a][e] = kv8_exp2(x[a][e]);
                    if constexpr (FIRST) l[a][e & 1] += w[a][e];
                    unit[a][e & 1] = pow2i(e_v) * KD_UNIT;
                }
            if (deep) {
                // y, of the step's own largest: it does not depend on M, so that the passes agree on who is whose
                constexpr int SPAN = KD_SPAN<FINE>;
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float s[2], m;
#pragma unroll
                        for (int e = 0; e < 2; ++e) s[e] = x[a][b + 2 * e] == -INFINITY ? -INFINITY : __fmul_rn(sc[a][b + 2 * e], by[a][b]);
                        m = fmaxf(s[0], s[1]);
#pragma unroll
                        for (int i = 4; i < 32; i <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
                        const float top = m == -INFINITY ? 0.f : floorf(m), up = KD_SHIFT + 1.f + SPAN * level, floor = -SPAN * (level + 1.f);
                        const float down = top - M[a][b] - up;   // M is a whole number: so is this
                        unit[a][b] *= m == -INFINITY || down < -126.f ? 0.f : pow2i((int)down);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float y = __fadd_rn(s[e], -top);
                            w[a][b + 2 * e] = y < floor || (!FIRST && y >= floor + SPAN) ? 0.f : kv8_exp2(y + up);
                            rest |= y < floor && x[a][b + 2 * e] > KD_SHIFT - KD_LAST;
                        }
                    }
                rest = __any_sync(0xffffffffu, rest);
            }
            // V of positions that not every token sees: their bytes may be anything, and 0 * NaN is not 0
            uint32_t v[4][HD / 32];   // keys 2t, 2t + 1, 2t + 8, 2t + 9: dims g * HD / 8 ..
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 2 * t + (x & 1) + (x >> 1) * 8;
                if constexpr (HD == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(step + 16 * HD + kd_at<HD>(key, g));
                    v[x][0] = w.x; v[x][1] = w.y; v[x][2] = w.z; v[x][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(step + 16 * HD + kd_at<HD>(key, g >> 1) + (g & 1) * 8);
                    v[x][0] = w.x; v[x][1] = w.y;
                }
            }
            uint32_t seen_nan[4] = {0, 0, 0, 0};   // bytes of visible NaN, where some tokens see them and some do not
            if (!all) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = kb + 2 * t + (x & 1) + (x >> 1) * 8;
                    bool any = false;
                    for (int n = max(-p0, 0); n < row.n; ++n) any |= kv8_sees(p0 + n, j, p.window, p.sinks);
                    if (!any) {
#pragma unroll
                        for (int d = 0; d < HD / 32; ++d) v[x][d] = 0u;
                    } else if (row.n > 1) {
#pragma unroll
                        for (int d = 0; d < HD / 32; ++d)
                            seen_nan[x] |= ((v[x][d] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    }
                }
            }
            if (__any_sync(0xffffffffu, seen_nan[0] | seen_nan[1] | seen_nan[2] | seen_nan[3])) {
                // rare: take the NaN bytes out of the product; the columns of the tokens that see them become NaN.
                // nan_s: which of the 16 keys hold a NaN, by dim
                for (int d = lane; d < HD; d += 32) nan_s[warp][d] = 0u;
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int d = 0; d < HD / 32; ++d) {
                        uint32_t at = ((v[x][d] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        v[x][d] &= ~((at >> 7) * 0xFFu);
                        while (at) {
                            const int bit = __ffs(at) - 1;
                            at &= at - 1;
                            atomicOr(&nan_s[warp][g * (HD / 8) + 4 * d + bit / 8], 1u << (2 * t + (x & 1) + (x >> 1) * 8));
                        }
                    }
                __syncwarp();
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t sees = 0u;   // keys that this query row sees
                        for (int j = 0; j < 16; ++j)
                            if (pos[a][b] >= 0 && kv8_sees(pos[a][b], kb + j, p.window, p.sinks)) sees |= 1u << j;
#pragma unroll
                        for (int k = 0; k < NK; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (nan_s[warp][g * (HD / 8) + 2 * k + e] & sees) o[a][k][b + 2 * e] = __int_as_float(0x7FFFFFFF);
                    }
            }
            // O += P V.  The tensor core cuts what it adds to its accumulator off, towards 0: over hundreds of steps that
            // shows in fp32 (7e-6 after 450), so the steps are added up outside, rounded, and V's exponent joins there
            uint32_t ph[MT][2], pl[MT][2];   // the weights that f16 holds in full, in two parts
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float w0 = w[a][2 * b], w1 = w[a][2 * b + 1];
                    const uint32_t hi = pack_f16x2(w0, w1);
                    const float2 f = unpack_f16x2(hi);
                    ph[a][b] = transpose8x8(hi);
                    pl[a][b] = transpose8x8(FINE ? pack_f16x2((w0 - f.x) * KD_LOW, (w1 - f.y) * KD_LOW) : pack_f16x2(w0 - f.x, w1 - f.y));
                }
#pragma unroll
            for (int d = 0; d < HD / 32; ++d) {
                // words of four keys, four dims each -> pairs of keys for dims 0, 1 and 2, 3
                const uint32_t x01 = __byte_perm(v[0][d], v[1][d], 0x5140), x23 = __byte_perm(v[0][d], v[1][d], 0x7362);
                const uint32_t y01 = __byte_perm(v[2][d], v[3][d], 0x5140), y23 = __byte_perm(v[2][d], v[3][d], 0x7362);
                uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
                e4m3x4_to_f16(x01, a0, a1);
                e4m3x4_to_f16(y01, a2, a3);
                e4m3x4_to_f16(x23, c0, c1);
                e4m3x4_to_f16(y23, c2, c3);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(x, a0, a1, a2, a3, pl[a][0], pl[a][1]);
                    mma_f16(y, c0, c1, c2, c3, pl[a][0], pl[a][1]);
                    if constexpr (FINE) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] *= 1.f / KD_LOW;
                            y[e] *= 1.f / KD_LOW;
                        }
                    }
                    mma_f16(x, a0, a1, a2, a3, ph[a][0], ph[a][1]);
                    mma_f16(y, c0, c1, c2, c3, ph[a][0], ph[a][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[a][2 * d][e] = fmaf(x[e], unit[a][e & 1], o[a][2 * d][e]);
                        o[a][2 * d + 1][e] = fmaf(y[e], unit[a][e & 1], o[a][2 * d + 1][e]);
                    }
                }
            }
            return rest;
        };

        uint32_t far = 0;   // the steps with weights that wait: step i has bit i % 32 of lane i / 32 % 32
        for (int i = 0; i < mine; ++i) {
            copy_next();
            copy_wait<STAGES - 1>();   // step i's group is complete
            __syncwarp();              // for every lane's copies
            const bool now = i >> 5 == (min(ahead, mine) - 1) >> 5;   // of the 32 held, or of the 32 before
            const int there = __shfl_sync(0xffffffffu, now ? place : place_before, i & 31);
            const int e_k = __shfl_sync(0xffffffffu, now ? ke : ke_before, i & 31) - 127;
            const int e_v = __shfl_sync(0xffffffffu, now ? ve : ve_before, i & 31) - 127;
            if (there >= 0 && compute(std::true_type{}, i, i % STAGES, e_k, e_v, 0) && lane == (i >> 5 & 31)) far |= 1u << (i & 31);
            __syncwarp();              // the stage may be overwritten
        }
        check_scales();
        copy_wait<0>();
        // The weights that wait: their steps again, 32 at a time.  Within the loop above the code of this would cost every
        // step (the compiler no longer overlaps them: 32 rows x 32k 235 us, so 225)
        if (__any_sync(0xffffffffu, far))
            for (int first = 0; first < mine; first += 32) {
                const uint32_t marks = __shfl_sync(0xffffffffu, far, first >> 5 & 31);
                if (!marks) continue;
                next32(first);
                uint32_t rest = marks;
                int copied = 0, done = 0;
                auto copy_marked = [&]() {
                    if (rest) copy_step(__ffs(rest) - 1, copied++ % STAGES);
                    rest &= rest - 1;
                    copy_commit();
                };
#pragma unroll
                for (int x = 0; x < STAGES - 1; ++x) copy_marked();
                for (uint32_t m = marks; m; m &= m - 1) {
                    const int l = __ffs(m) - 1;
                    copy_marked();
                    copy_wait<STAGES - 1>();
                    __syncwarp();
                    const int there = __shfl_sync(0xffffffffu, place, l);
                    const int e_k = __shfl_sync(0xffffffffu, ke, l) - 127, e_v = __shfl_sync(0xffffffffu, ve, l) - 127;
                    const int stage = done++ % STAGES;
                    if (there >= 0)
                        for (int level = 1; compute(std::false_type{}, first + l, stage, e_k, e_v, level); ++level) {}
                    __syncwarp();   // the stage may be overwritten
                }
                copy_wait<0>();
            }
        __syncthreads();   // every warp is done with its ring

        // join the warps: the largest maximum, then sums in warp order
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[a][b] += __shfl_xor_sync(0xffffffffu, l[a][b], x);
                if (g == 0) {
                    m_s[warp][a * 8 + 2 * t + b] = M[a][b] == KD_NONE ? -INFINITY : M[a][b];
                    l_s[warp][a * 8 + 2 * t + b] = l[a][b];
                }
            }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int k = 0; k < NK; ++k)   // dims g * HD / 8 + 2 k, + 1
                    *reinterpret_cast<float2*>(&o_s[warp][a * 8 + 2 * t + b][g * (HD / 8) + 2 * k]) =
                        make_float2(o[a][k][b], o[a][k][b + 2]);
        __syncthreads();
        const bool whole = i0 == 0 && i1 == tl.n;
        float* slots = p.ws;
        float* slot = slots + ((size_t)blockIdx.x * 2 + (u == u_begin ? 0 : 1)) * kd_slot_floats<HD, MT>();
        auto put = [&](int m, int d, float sum, const float (&y)[4]) {
            const float inv = sum == 0.f ? 0.f : 1.f / (sum * KD_UNIT);   // nothing seen: zeros
            const int n = p.by_group.of(m);
            T* dst = static_cast<T*>(p.out) + (row.t0 + n) * p.out_stride + (h * G + m - n * G) * HD + d;
            if constexpr (FINE) *reinterpret_cast<float4*>(dst) = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv));
        };
        for (int x = tid; x < nq * (HD / 4); x += 32 * W) {
            const int m = x / (HD / 4), d = (x % (HD / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, m_s[w][m]);
            float sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = m_s[w][m] == -INFINITY ? 0.f : kv8_exp2(m_s[w][m] - top);
                const float4 v = *reinterpret_cast<const float4*>(&o_s[w][m][d]);
                if (m_s[w][m] == -INFINITY && l_s[w][m] == 0.f) continue;   // nothing seen by this warp
                sum += l_s[w][m] * f;
                y[0] += v.x * f; y[1] += v.y * f; y[2] += v.z * f; y[3] += v.w * f;
            }
            if (whole) {
                put(m, d, sum, y);
            } else {
                *reinterpret_cast<float4*>(slot + m * HD + d) = make_float4(y[0], y[1], y[2], y[3]);
                if (d == 0) {
                    slot[MT * 8 * HD + m] = top;
                    slot[MT * 8 * (HD + 1) + m] = sum;
                }
            }
        }
        if (!whole) {
            // the last CTA of this row and head joins the pieces' parts, in their order
            __syncthreads();
            if (tid == 0) {
                __threadfence();   // the CTA's parts, before its arrival is counted
                last_s = atomicAdd(p.counters + r * c.Hkv + h, 1) == c1 - c0;
                __threadfence();
            }
            __syncthreads();
            if (last_s) {
                const bool second = !cut.own && cut.begin(c0) != u - i0;   // piece c0 had other work before
                // 8 columns of a query row are an item; where there are fewer items than threads, several threads share
                // an item's parts, a run of them each
                const int items = nq * (HD / 8), teams = max(32 * W / items, 1), run = (c1 - c0 + teams) / teams;
                float* shared = reinterpret_cast<float*>(kd_raw);   // [teams][items][12]: the warps' results are not needed any more
                for (int x = tid; x < items * teams; x += 32 * W) {
                    const int team = x / items, item = x - team * items, m = item / (HD / 8), d = (item % (HD / 8)) * 8;
                    const int from = c0 + team * run, to = min(from + run - 1, c1);
                    float top = -INFINITY, sum = 0.f, y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = 0.f;
                    constexpr int B = 6;   // parts read at once
                    for (int q0 = from; q0 <= to; q0 += B) {
                        float mm[B], ll[B], big = top;
                        float4 v[B][2];
#pragma unroll
                        for (int k = 0; k < B; ++k) {
                            const int q = min(q0 + k, to);
                            const float* part = slots + ((size_t)q * 2 + (q == c0 && second ? 1 : 0)) * kd_slot_floats<HD, MT>();
                            mm[k] = __ldcg(part + MT * 8 * HD + m);
                            ll[k] = __ldcg(part + MT * 8 * (HD + 1) + m);
                            v[k][0] = __ldcg(reinterpret_cast<const float4*>(part + m * HD + d));
                            v[k][1] = __ldcg(reinterpret_cast<const float4*>(part + m * HD + d) + 1);
                        }
#pragma unroll
                        for (int k = 0; k < B; ++k) big = fmaxf(big, mm[k]);
                        const float f = top == -INFINITY ? 0.f : kv8_exp2(top - big);
                        sum *= f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] *= f;
                        top = big;
#pragma unroll
                        for (int k = 0; k < B; ++k) {
                            if (q0 + k > to || (mm[k] == -INFINITY && ll[k] == 0.f)) continue;   // nothing seen there
                            const float e = mm[k] == -INFINITY ? 0.f : kv8_exp2(mm[k] - big);
                            sum += ll[k] * e;
                            y[0] += v[k][0].x * e; y[1] += v[k][0].y * e; y[2] += v[k][0].z * e; y[3] += v[k][0].w * e;
                            y[4] += v[k][1].x * e; y[5] += v[k][1].y * e; y[6] += v[k][1].z * e; y[7] += v[k][1].w * e;
                        }
                    }
                    float4* mine_s = reinterpret_cast<float4*>(shared + (team * items + item) * 12);
                    mine_s[0] = make_float4(y[0], y[1], y[2], y[3]);
                    mine_s[1] = make_float4(y[4], y[5], y[6], y[7]);
                    mine_s[2] = make_float4(top, sum, 0.f, 0.f);
                }
                __syncthreads();
                for (int x = tid; x < items; x += 32 * W) {
                    const int m = x / (HD / 8), d = (x % (HD / 8)) * 8;
                    float top = -INFINITY, sum = 0.f, y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = 0.f;
                    for (int w = 0; w < teams; ++w) top = fmaxf(top, shared[(w * items + x) * 12 + 8]);
                    for (int w = 0; w < teams; ++w) {
                        const float* o = shared + (w * items + x) * 12;
                        if (o[8] == -INFINITY && o[9] == 0.f) continue;   // nothing seen there
                        const float e = o[8] == -INFINITY ? 0.f : kv8_exp2(o[8] - top);
                        sum += o[9] * e;
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] += o[k] * e;
                    }
                    put(m, d, sum, reinterpret_cast<const float(&)[4]>(y[0]));
                    put(m, d + 4, sum, reinterpret_cast<const float(&)[4]>(y[4]));
                }
                if (tid == 0) p.counters[r * c.Hkv + h] = 0;   // for the next call
            }
        }
        __syncthreads();   // the shared buffers are free again
        u += cut.own ? 1 : i1 - i0;
    }
    // not earlier: the next kernel's blocks would take places that this grid, which is one wave, counts on
    pdl_trigger();
}

// Tokens of a row that a launch takes, and the launches.  A prompt kernel's CTA has 256 query rows, so drafts of a large
// batch leave most of it idle: there the stream of K and V, read two or three times, may be shorter.  It is cut evenly
// where the lengths differ, the prompt kernel's time is the longest row's.  Measured, here and by the prompt kernel, 4
// query heads a K/V head, 8 tokens (two launches), rows of equal and of unequal lengths: 16 rows x 32k bf16 542 and 569,
// 333 and 564, fp32 610 and 927, 373 and 906; 32 rows x 4k bf16 182 and 161, 124 and 143, fp32 202 and 259, 138 and 220;
// 8 rows x 8k, where the prompt kernel splits the positions over the SMs, bf16 115 and 85, 74 and 81, fp32 128 and 133,
// 82 and 131.  12 tokens (three), 16 rows x 32k: bf16 814 and 577, 494 and 573, fp32 916 and 930, 555 and 909.  With one
// row x 8k it is as fast as one launch here (8 tokens 25 us, 4 tokens 26), and for short caches a launch is what counts
int decode_tokens(const Kv8Attend& p) { return p.b.max_new * p.G <= 16 ? p.b.max_new : 16 / p.G; }
int decode_launches(const Kv8Attend& p, int num_sms) {
    const int each = decode_tokens(p);
    if (each == p.b.max_new) return 1;
    const bool fine = p.dtype == W_F32;
    if (each == 0 || p.b.max_new > (fine ? 3 : 2) * each) return 0;
    const long long cap = (long long)p.c.ppr * p.c.page, win = (long long)p.window + p.sinks + p.b.max_new;
    const long long heads = (long long)p.c.rows * p.c.Hkv;
    const int n = (p.b.max_new + each - 1) / each;
    return (win < cap ? win : cap) >= 2048 && (fine && n == 2 ? 3 : 2) * heads >= num_sms ? n : 0;
}
int decode_sets(const Kv8Attend& p) { return (decode_tokens(p) * p.G + 7) / 8; }

// one CTA for each place on the GPU, but no more than there can be steps
int decode_grid(const Kv8Attend& p, int num_sms) {
    const long long steps = (long long)p.c.rows * p.c.Hkv * (((long long)p.c.ppr * p.c.page + KD_STEP - 1) / KD_STEP);
    const int most = num_sms * KdShared<128, 1>::CTAS;
    return (int)(steps < most ? steps : most);
}

template <int HD, int MT, bool FINE>
cudaError_t launch(const Kv8Attend& p, int num_sms, cudaStream_t s) {
    using S = KdShared<HD, MT>;
    static OncePerDevice raised;
    cudaError_t e = raised.run([] {
        return cudaFuncSetAttribute((const void*)&k_kv8_decode<HD, MT, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(decode_grid(p, num_sms));
    cfg.blockDim = dim3(32 * S::W);
    cfg.dynamicSmemBytes = S::BYTES;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv8_decode<HD, MT, FINE>, p);
}

}  // namespace

bool kv8_decode_takes(const Kv8Attend& p, int num_sms) { return decode_launches(p, num_sms) > 0; }

size_t kv8_decode_floats(const Kv8Attend& p, int num_sms) {
    return (size_t)decode_grid(p, num_sms) * 2 * decode_sets(p) * 8 * (p.c.hd + 2);
}

cudaError_t kv8_decode_launch(const Kv8Attend& p, int num_sms, cudaStream_t s) {
    const int each = decode_tokens(p);
    if (!p.take && each < p.b.max_new) {
        cudaError_t e = cudaSuccess;
        Kv8Attend some = p;
        some.take = each;
        for (; some.skip < p.b.max_new && e == cudaSuccess; some.skip += each) e = kv8_decode_launch(some, num_sms, s);
        return e;
    }
    const bool two = decode_sets(p) == 2, fine = p.dtype == W_F32;
    if (p.c.hd == 128) {
        if (fine) return two ? launch<128, 2, true>(p, num_sms, s) : launch<128, 1, true>(p, num_sms, s);
        return two ? launch<128, 2, false>(p, num_sms, s) : launch<128, 1, false>(p, num_sms, s);
    }
    if (fine) return two ? launch<64, 2, true>(p, num_sms, s) : launch<64, 1, true>(p, num_sms, s);
    return two ? launch<64, 2, false>(p, num_sms, s) : launch<64, 1, false>(p, num_sms, s);
}

}  // namespace gd
