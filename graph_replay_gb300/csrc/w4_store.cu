// w4_store.cu -- storing a matrix in 4 bits, and reading it back.
//
// quantize: over each group of 32, 64 or 128 columns of a row
//   s = bf16(max |w| / 7),  q = w / s to the nearest whole number (ties to even),
// so |q| <= 7; s < 2^-100: s = 0 and q = 0; a NaN or an infinity in the group:
// s = NaN.  A lane holds 8 columns, so a group is 4, 8 or 16 lanes of a warp and
// its largest value needs no shared memory.  The quotient is found without a
// division: q0 = rint(w * (1 / s)) is at most one off, and w - q0 s is exact in one
// fused multiply-add, so comparing it with s / 2 decides every case, ties too.
// Bound by memory: 2 or 4 bytes a weight read, 0.5 + 2 / group written.
#include "w4.cuh"

namespace gd {

namespace {

constexpr int QT = 256;   // threads

template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&v)[8]) {
    if (F32) {
        const uint4 a = ld_stream16(reinterpret_cast<const float*>(p) + i);
        const uint4 b = ld_stream16(reinterpret_cast<const float*>(p) + i + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        Elem<__nv_bfloat16>::unpack(ld_stream16(reinterpret_cast<const __nv_bfloat16*>(p) + i), v);
    }
}

__device__ __forceinline__ uint32_t code8(const float (&v)[8], float s, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q = rintf(v[i] * inv);
        const float r = fmaf(-q, s, v[i]);           // exact: |r| < s
        const float d = 2.0f * fabsf(r) - s;         // exact in sign: both are multiples of one power of two
        const float to = r > 0.0f ? 1.0f : -1.0f;
        const bool odd = (int)q & 1;
        if (d > 0.0f || (d == 0.0f && odd)) q += to;
        w |= ((uint32_t)(int)q & 15u) << (4 * i);
    }
    return w;
}

// one item: 8 columns; n * k / 8 items in all, items of a row side by side
template <bool F32>
__global__ void __launch_bounds__(QT) k_w4_quantize(const void* __restrict__ src, long long stride, uint32_t* __restrict__ codes,
                                                    __nv_bfloat16* __restrict__ scales, int items, FastDiv k8, int lanes) {
    const unsigned step = gridDim.x * QT;   // items < 2^31: no sum below wraps
    const int lane = threadIdx.x & 31;
    for (unsigned i0 = blockIdx.x * QT + threadIdx.x; i0 - lane < (unsigned)items; i0 += step) {
        const bool live = i0 < (unsigned)items;
        const int i = live ? (int)i0 : items - 1;
        const int row = k8.of(i);
        const int c = i - row * (int)k8.d;
        float v[8];
        load8<F32>(src, (size_t)row * stride + (size_t)c * 8, v);
        uint32_t top = 0;   // the bits of |x| order like the values, with infinity and NaN above them
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        for (int o = 1; o < lanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool bad = top >= 0x7f800000u;
        __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.0f));
        float s = __bfloat162float(sb);
        const bool none = bad || s < 7.8886090522101181e-31f;   // 2^-100
        if (none) {
            sb = __ushort_as_bfloat16(bad ? 0x7fc0 : 0);
            s = 1.0f;
        }
        uint32_t w = 0;
        if (!none) w = code8(v, s, __frcp_rn(s));
        if (live) {
            codes[i] = w;
            if (lane % lanes == 0) scales[i / lanes] = sb;   // groups of all rows follow one another
        }
    }
}

// code * scale in fp32 (exact), rounded once where the values are bf16
template <bool F32>
__global__ void __launch_bounds__(QT) k_w4_values(const uint32_t* __restrict__ codes, const __nv_bfloat16* __restrict__ scales,
                                                  void* __restrict__ dst, long long stride, int items, FastDiv k8, int lanes) {
    const unsigned step = gridDim.x * QT;
    for (unsigned i = blockIdx.x * QT + threadIdx.x; i < (unsigned)items; i += step) {
        const int row = k8.of((int)i);
        const int c = (int)i - row * (int)k8.d;
        const uint32_t w = codes[i];
        const float s = __bfloat162float(scales[i / lanes]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)((int)(w << (28 - 4 * e)) >> 28) * s;
        const size_t at = (size_t)row * stride + (size_t)c * 8;
        if (F32) {
            float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(dst) + at);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint4 o;
            uint32_t* u = &o.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(dst) + at) = o;
        }
    }
}

int grid_for(int items, int num_sms) {
    const int blocks = (items - 1) / QT + 1;
    return blocks < num_sms * 8 ? blocks : num_sms * 8;
}

}  // namespace

cudaError_t w4_quantize_launch(const W4Matrix& w, const void* src, long long stride, bool f32, int num_sms, cudaStream_t s) {
    const int items = w.n * (w.k / 8);
    const int grid = grid_for(items, num_sms);
    uint32_t* codes = reinterpret_cast<uint32_t*>(const_cast<void*>(w.codes));
    __nv_bfloat16* scales = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(w.scales));
    if (f32) k_w4_quantize<true><<<grid, QT, 0, s>>>(src, stride, codes, scales, items, FastDiv((unsigned)(w.k / 8)), w.group / 8);
    else k_w4_quantize<false><<<grid, QT, 0, s>>>(src, stride, codes, scales, items, FastDiv((unsigned)(w.k / 8)), w.group / 8);
    return cudaGetLastError();
}

cudaError_t w4_values_launch(const W4Matrix& w, void* dst, long long stride, bool f32, int num_sms, cudaStream_t s) {
    const int items = w.n * (w.k / 8);
    const int grid = grid_for(items, num_sms);
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(w.codes);
    const __nv_bfloat16* scales = reinterpret_cast<const __nv_bfloat16*>(w.scales);
    if (f32) k_w4_values<true><<<grid, QT, 0, s>>>(codes, scales, dst, stride, items, FastDiv((unsigned)(w.k / 8)), w.group / 8);
    else k_w4_values<false><<<grid, QT, 0, s>>>(codes, scales, dst, stride, items, FastDiv((unsigned)(w.k / 8)), w.group / 8);
    return cudaGetLastError();
}

}  // namespace gd
