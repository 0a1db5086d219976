// kv8_append.cu -- new tokens' K and V into the 8-bit cache.
//
// For each block of positions and K/V head that new tokens enter: e is the
// least exponent with max |x| <= 448 * 2^e over the new finite values (448 is
// e4m3's largest), at least the block's exponent if it holds earlier positions;
// x is stored as e4m3(x * 2^-e), round to nearest even.  Where e grew, the
// earlier positions' bytes are rounded again at the new exponent: a shift by a
// power of two, which loses bits only below 2^-6, e4m3's least normal value.
// NaN, infinities and what 2^KV8_EXP_MAX cannot hold are stored as NaN.
//
// One CTA takes one block of one head of K or of V, so a block's maximum needs
// no memory between CTAs and every byte is written once.  A thread keeps its
// values in registers between the maximum and the rounding: the input is read
// once.  Bound: those reads and writes, and close behind them the issue of
// instructions (bf16 141 MB in 26.9 us, 5.25 TB/s, fp32 235 MB in 40 us, 5.9 TB/s); for a single token three
// dependent trips to memory (1.9 us).
#include "kv8.cuh"

namespace gd {

namespace {

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.402823466e38f; }

// 8 values as they came from memory, until they are needed: half the registers for bf16
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ld_stream16(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        constexpr int N = Elem<T>::VEC;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            float x[N];
            Elem<T>::unpack(w[i], x);
#pragma unroll
            for (int k = 0; k < N; ++k) f[i * N + k] = x[k];
        }
    }
};

// largest magnitude, infinities among them; a NaN never wins fmaxf or __hmax2
__device__ __forceinline__ float top_of(const Raw8<float>& v, float top) {
    float x[8];
    v.values(x);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
    return top;
}
__device__ __forceinline__ float top_of(const Raw8<__nv_bfloat16>& v, float top) {   // two at a time
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v.w[0]);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(x[0]), __habs2(x[1])), __hmax2(__habs2(x[2]), __habs2(x[3])));
    return fmaxf(top, fmaxf(__low2float(m), __high2float(m)));
}
// v * 2^-e.  bf16 has fp32's exponents, so two at a time are as exact: only what is far below e4m3's least step is lost
__device__ __forceinline__ void scale(Raw8<float>& v, float inv, float (&f)[8]) {
    v.values(f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= inv;
}
__device__ __forceinline__ void scale(Raw8<__nv_bfloat16>& v, float inv, float (&f)[8]) {
    __nv_bfloat162* x = reinterpret_cast<__nv_bfloat162*>(&v.w[0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __hmul2(x[k], __float2bfloat162_rn(inv));
    v.values(f);
}
// largest of the CTA's values; `tops` holds a slot for each warp and is free when the CTA enters
__device__ __forceinline__ float cta_max(float top, float* tops) {
    top = warp_max(top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    top = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) top = fmaxf(top, tops[w]);
    return top;
}

// grid (blocks a row may touch, 2 * Hkv, rows); NCH: chunks of 8 values a thread may hold
template <typename T, int NCH>
__global__ void k_kv8_append(const Kv8Append p) {
    __shared__ float tops[2][8];
    const int r = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1, tid = threadIdx.x;
    const Kv8Cache& c = p.c;
    Kv8Row row;
    if (!kv8_row(p.b, c.ppr * c.page, r, &row)) return;
    const int first = max(row.len - row.n, 0);   // tokens before position 0 have no place
    const int b0 = ((first >> c.block_log2) + (int)blockIdx.x) << c.block_log2;
    if (b0 >= row.len || row.n == 0) return;
    const int lo = max(first, b0), hi = min(row.len, b0 + c.block);
    const long long stride = which ? p.v_stride : p.k_stride;
    const T* src = static_cast<const T*>(which ? p.v : p.k) + (row.t0 + lo - (row.len - row.n)) * stride + (size_t)h * c.hd;
    const int log2_per = c.hd == 128 ? 4 : 3, chunks = (hi - lo) << log2_per;
    // the values are on their way before the page's id is known
    Raw8<T> v[NCH];
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
        const int i = tid + u * blockDim.x;
        if (i < chunks) v[u].load(src + (i >> log2_per) * stride + (i & ((1 << log2_per) - 1)) * 8);
    }
    const int slot = c.by_page.of(b0), off = b0 - slot * c.page;
    const int page = kv8_page(c, p.b.err, r, slot);
    if (page < 0) return;
    const size_t head = (size_t)page * c.Hkv + h;
    uint8_t* dst = (which ? c.v : c.k) + (head * c.page + off) * c.hd;
    uint8_t* sc = (which ? c.vs : c.ks) + head * (c.page >> c.block_log2) + (off >> c.block_log2);
    const int held = lo - b0;   // earlier positions in the block
    const int had = held ? (int)*sc - 127 : -1000;

    // The kernel's instructions set its time as much as its bytes do, so infinities, NaN and what the largest exponent
    // cannot hold cost the other blocks one compare: the plain maximum tells whether the block has any but NaN
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < NCH; ++u)
        if (tid + u * (int)blockDim.x < chunks) top = top_of(v[u], top);
    const float all = top = cta_max(top, tops[0]);   // and every thread has read the old exponent
    if (!finite_f(all)) {   // again, over the finite values
        top = 0.f;
#pragma unroll
        for (int u = 0; u < NCH; ++u)
            if (tid + u * (int)blockDim.x < chunks) {
                float x[8];
                v[u].values(x);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (finite_f(x[k])) top = fmaxf(top, fabsf(x[k]));
            }
        top = cta_max(top, tops[1]);
    }
    const int e = max(kv8_exponent(top), had);
    // a caller's own scale bytes go beyond what append writes: 118 keeps the limit finite, 126 the factor normal
    const bool beyond = all > 448.f * pow2i(min(e, 118)) || e > 126;
    if (tid == 0) *sc = (uint8_t)(e + 127);
    const float inv = pow2i(-min(e, 126));
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
        const int i = tid + u * blockDim.x;
        if (i >= chunks) continue;
        float x[8];
        scale(v[u], inv, x);
        if (beyond) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[k] *= pow2i(min(126 - e, 0));
                if (!(fabsf(x[k]) <= 448.f)) x[k] = __int_as_float(0x7FFFFFFF);
            }
        }
        *reinterpret_cast<uint2*>(dst + (size_t)held * c.hd + (size_t)i * 8) =
            make_uint2(f32_to_e4m3x4(x[0], x[1], x[2], x[3]), f32_to_e4m3x4(x[4], x[5], x[6], x[7]));
    }
    if (held && e > had) {
        const float f = pow2i(max(had - e, -60));
        for (int i = tid; i < held << log2_per; i += blockDim.x) {
            uint2* q = reinterpret_cast<uint2*>(dst) + i;
            float a[4], b[4];
            e4m3x4_to_f32(q->x, a);
            e4m3x4_to_f32(q->y, b);
            *q = make_uint2(f32_to_e4m3x4(a[0] * f, a[1] * f, a[2] * f, a[3] * f),
                            f32_to_e4m3x4(b[0] * f, b[1] * f, b[2] * f, b[3] * f));
        }
    }
}

template <typename T>
cudaError_t launch(const Kv8Append& p, cudaStream_t s) {
    const int span = p.b.max_new < p.c.block ? p.b.max_new : p.c.block;   // tokens of one block
    const int chunks = span * (p.c.hd / 8);
    // Few threads with many loads each: a CTA waits most of its life, so what counts is the bytes that an SM's 2048
    // threads have under way (4 prompts of up to 8191 tokens, bf16: 128 threads 27 us, 64 or 256 threads 29; fp32: 128 or
    // 256 threads 40)
    const int threads = chunks <= 64 ? 64 : sizeof(T) == 2 ? 128 : 256;
    const dim3 grid((p.b.max_new + p.c.block - 2) / p.c.block + 1, 2 * p.c.Hkv, p.c.rows);
    if (chunks <= threads) k_kv8_append<T, 1><<<grid, threads, 0, s>>>(p);
    else if (chunks <= 2 * threads) k_kv8_append<T, 2><<<grid, threads, 0, s>>>(p);
    else if (chunks <= 4 * threads) k_kv8_append<T, 4><<<grid, threads, 0, s>>>(p);
    else if (chunks <= 8 * threads) k_kv8_append<T, 8><<<grid, threads, 0, s>>>(p);
    else if constexpr (sizeof(T) == 2) k_kv8_append<T, 16><<<grid, threads, 0, s>>>(p);   // 128 positions of 128 dims
    else return cudaErrorInvalidValue;   // not reached: 256 threads hold a block of fp32
    return cudaGetLastError();
}

}  // namespace

cudaError_t kv8_append_launch(const Kv8Append& p, cudaStream_t s) {
    return p.dtype == W_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace gd
