// w4_store.cu -- storing a matrix in 4 bits, and reading it back.
//
// quantize: over each group of 32, 64 or 128 columns of a row
//   s = bf16(max |w| / 7),  q = w / s to the nearest whole number (ties to even),
// so |q| <= 7; s < 2^-100: s = 0 and q = 0; a NaN or an infinity in the group:
// s = NaN.  A lane holds 16 columns, so a group is 2, 4 or 8 lanes of a warp and
// its largest value needs no shared memory.  The quotient is found without a
// division: w * (1 / s) to the nearest whole number is at most one off, and w - q s is
// exact in one fused multiply-add, so comparing it with s / 2 decides every case, ties
// too.
// Bound by memory, 2 or 4 bytes a weight read, 0.5 + 2 / group written, where the weights
// are fp32: 14336 x 4096 in 47.6 us, 5.6 TB/s (a copy: 6.8).  bf16 ones take 42.5 us, 3.5
// TB/s: there the border of each code, about a dozen instructions a weight, takes as long
// as the bytes (two would do where the weight has 8 bits: w / s is never nearer to a border
// than 2^-10 without being on it).  Reading back: 28.9 us to bf16 (5.1 TB/s), 64 to fp32 (4.1),
// where a lane's two stores are 32 bytes side by side, so each of a warp's covers half of the
// sectors that it touches.
// With conversions between integers and floats and 8 columns a lane, storing and reading
// back in bf16 took 110 us together; 71 now.
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

// 1.5 * 2^23: a sum with it is a whole number in fp32 (to the nearest, ties to even), whose low bits are the number's in
// two's complement.  So no conversion between integers and floats is needed, which run at a quarter of the rate
constexpr float MAGIC = 12582912.0f;

__device__ __forceinline__ uint32_t code8(const float (&v)[8], float s, float inv) {
    const float half = 0.5f * s;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float m = fmaf(v[i], inv, MAGIC);            // of w * (1 / s): right, or one off next to a border
        const float r = fmaf(MAGIC - m, s, v[i]);    // w - q s, exact
        // beyond half a step, or on the border at an odd code: one further
        const bool odd = __float_as_uint(m) & 1u;
        if (fabsf(r) > half || (fabsf(r) == half && odd)) m += copysignf(1.0f, r);
        w |= (__float_as_uint(m) & 15u) << (4 * i);
    }
    return w;
}

// one item: 16 columns (so that a group's scale is found by few lanes); n * k / 16 items in all, items of a row side by side
template <bool F32>
__global__ void __launch_bounds__(QT) k_w4_quantize(const void* __restrict__ src, long long stride, uint2* __restrict__ codes,
                                                    __nv_bfloat16* __restrict__ scales, int items, FastDiv k16, int lanes) {
    const unsigned step = gridDim.x * QT;   // items < 2^31: no sum below wraps
    const int lane = threadIdx.x & 31;
    for (unsigned first = blockIdx.x * QT + threadIdx.x; first - lane < (unsigned)items; first += step) {
        const int i = (int)min(first, (unsigned)items - 1u);
        const int row = k16.of(i);
        const size_t at = (size_t)row * stride + (size_t)(i - row * (int)k16.d) * 16;
        float a[8], b[8];
        load8<F32>(src, at, a);
        load8<F32>(src, at + 8, b);
        uint32_t top = 0;   // the bits of |x| order like the values, with infinity and NaN above them
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, max(__float_as_uint(a[e]) & 0x7fffffffu, __float_as_uint(b[e]) & 0x7fffffffu));
        for (int o = 1; o < lanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool bad = top >= 0x7f800000u;
        __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.0f));
        const float s = __bfloat162float(sb);
        const bool none = bad || s < 7.8886090522101181e-31f;   // 2^-100
        const float inv = __frcp_rn(none ? 1.0f : s);
        const uint32_t wa = code8(a, none ? 1.0f : s, inv), wb = code8(b, none ? 1.0f : s, inv);
        if (first < (unsigned)items) {
            codes[i] = none ? make_uint2(0u, 0u) : make_uint2(wa, wb);
            // groups of all rows follow one another
            if ((lane & (lanes - 1)) == 0) scales[(unsigned)i / (unsigned)lanes] = none ? __ushort_as_bfloat16(bad ? 0x7fc0 : 0) : sb;
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
        const float s = __bfloat162float(scales[i / (unsigned)lanes]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)   // 2^23 + (q + 8), less 2^23 + 8
            v[e] = (__uint_as_float(((w >> (4 * e) & 15u) ^ 0x4b000008u)) - 8388616.0f) * s;
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
    const int items = w.n * (w.k / 16), grid = grid_for(items, num_sms), lanes = w.group / 16;
    const FastDiv k16((unsigned)(w.k / 16));
    uint2* codes = reinterpret_cast<uint2*>(const_cast<void*>(w.codes));
    __nv_bfloat16* scales = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(w.scales));
    if (f32) k_w4_quantize<true><<<grid, QT, 0, s>>>(src, stride, codes, scales, items, k16, lanes);
    else k_w4_quantize<false><<<grid, QT, 0, s>>>(src, stride, codes, scales, items, k16, lanes);
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
