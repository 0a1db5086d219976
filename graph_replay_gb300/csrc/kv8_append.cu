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
// once.
#include "kv8.cuh"

namespace gd {

namespace {

constexpr int KV8_EXP_MIN = -40, KV8_EXP_MAX = 60;

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.402823466e38f; }

// least e with top <= 448 * 2^e; 448 = 1.75 * 2^8
__device__ __forceinline__ int kv8_exponent(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, KV8_EXP_MIN), KV8_EXP_MAX);
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), f);
}

// grid (blocks a row may touch, 2 * Hkv, rows); NCH: chunks of 8 values a thread may hold
template <typename T, int NCH>
__global__ void k_kv8_append(const Kv8Append p) {
    __shared__ float tops[32];
    const int r = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1, tid = threadIdx.x;
    const Kv8Cache& c = p.c;
    Kv8Row row;
    if (!kv8_row(p.b, c.ppr * c.page, r, &row)) return;
    const int first = max(row.len - row.n, 0);   // tokens before position 0 have no place
    const int b0 = (first / c.block + (int)blockIdx.x) * c.block;
    if (b0 >= row.len || row.n == 0) return;
    const int lo = max(first, b0), hi = min(row.len, b0 + c.block);
    const int page = kv8_page(c, p.b.err, r, b0 / c.page);
    if (page < 0) return;
    const int off = b0 % c.page;
    const size_t head = (size_t)page * c.Hkv + h;
    uint8_t* dst = (which ? c.v : c.k) + (head * c.page + off) * c.hd;
    uint8_t* sc = (which ? c.vs : c.ks) + head * (c.page / c.block) + off / c.block;
    const long long stride = which ? p.v_stride : p.k_stride;
    const T* src = static_cast<const T*>(which ? p.v : p.k) + (row.t0 + lo - (row.len - row.n)) * stride + (size_t)h * c.hd;
    const int per = c.hd / 8, chunks = (hi - lo) * per;

    float v[NCH][8];
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
        const int i = tid + u * blockDim.x;
        if (i < chunks) load8(src + (i / per) * stride + (i % per) * 8, v[u]);
    }
#pragma unroll
    for (int u = 0; u < NCH; ++u)
        if (tid + u * (int)blockDim.x < chunks)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (finite_f(v[u][k])) top = fmaxf(top, fabsf(v[u][k]));
    top = warp_max(top);
    if ((tid & 31) == 0) tops[tid >> 5] = top;
    __syncthreads();
    top = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) top = fmaxf(top, tops[w]);
    int e = kv8_exponent(top);
    const int held = lo - b0;   // earlier positions in the block
    const int had = held ? (int)*sc - 127 : e;
    e = max(e, had);
    const float inv = pow2i(-min(e, 126));
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
        const int i = tid + u * blockDim.x;
        if (i >= chunks) continue;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = v[u][k] * inv;
            if (!(fabsf(x[k]) <= 448.f)) x[k] = __int_as_float(0x7FFFFFFF);
        }
        *reinterpret_cast<uint2*>(dst + (size_t)held * c.hd + (size_t)i * 8) =
            make_uint2(f32_to_e4m3x4(x[0], x[1], x[2], x[3]), f32_to_e4m3x4(x[4], x[5], x[6], x[7]));
    }
    if (e > had) {
        const float f = pow2i(max(had - e, -60));
        for (int i = tid; i < held * per; i += blockDim.x) {
            uint2* q = reinterpret_cast<uint2*>(dst) + i;
            float a[4], b[4];
            e4m3x4_to_f32(q->x, a);
            e4m3x4_to_f32(q->y, b);
            *q = make_uint2(f32_to_e4m3x4(a[0] * f, a[1] * f, a[2] * f, a[3] * f),
                            f32_to_e4m3x4(b[0] * f, b[1] * f, b[2] * f, b[3] * f));
        }
    }
    __syncthreads();   // every thread has read the old exponent
    if (tid == 0) *sc = (uint8_t)(e + 127);
}

template <typename T>
cudaError_t launch(const Kv8Append& p, cudaStream_t s) {
    const int span = p.b.max_new < p.c.block ? p.b.max_new : p.c.block;   // tokens of one block
    const int chunks = span * (p.c.hd / 8);
    const int threads = chunks <= 64 ? 64 : 256;
    const dim3 grid((p.b.max_new + p.c.block - 2) / p.c.block + 1, 2 * p.c.Hkv, p.c.rows);
    if (chunks <= threads) k_kv8_append<T, 1><<<grid, threads, 0, s>>>(p);
    else if (chunks <= 2 * threads) k_kv8_append<T, 2><<<grid, threads, 0, s>>>(p);
    else if (chunks <= 4 * threads) k_kv8_append<T, 4><<<grid, threads, 0, s>>>(p);
    else k_kv8_append<T, 8><<<grid, threads, 0, s>>>(p);   // 128 positions of 128 dims
    return cudaGetLastError();
}

}  // namespace

cudaError_t kv8_append_launch(const Kv8Append& p, cudaStream_t s) {
    return p.dtype == W_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace gd
