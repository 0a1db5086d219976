// w4.cuh -- device helpers shared by the kernels of the 4-bit weights.
//
// A stored matrix [n, k] is codes [n, k / 2] (two's complement, -8 .. 7, column
// 2i in the low half of byte i) and bf16 scales [n, k / group].  A 32-bit word
// holds eight columns; its halves hold columns 0-3 and 4-7, so one AND gives the
// pair (j, j + 4) in the two halves of a register.
//
// Codes become fp16 by placing them in the mantissa of 1024 (low position, steps
// of 1) or of 1024 with steps of 16 (next position): with bit 3 turned over the
// half reads 1024 + (q + 8) or 1024 + 16 (q + 8), and one exact half-precision
// operation leaves q.  All of it is exact.
#pragma once
#include <cuda_fp16.h>
#include "common.cuh"
#include "internal.h"

namespace gd {

__device__ __forceinline__ uint32_t w4_hsub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t w4_hfma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t w4_hmul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a & mask) ^ c in one instruction
template <uint32_t MASK>
__device__ __forceinline__ uint32_t w4_and_xor(uint32_t a, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "n"(MASK), "r"(c));
    return r;
}
// constants that stay in registers: as immediates they would cost an instruction more at each use
struct W4Const {
    uint32_t low, high, part, less;            // 1032, the pattern of the next position, 1 / 16, -72, in both halves
    __device__ __forceinline__ W4Const() {
        asm volatile("mov.b32 %0, 0x64086408;" : "=r"(low));
        asm volatile("mov.b32 %0, 0x64806480;" : "=r"(high));
        asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(part));
        asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(less));
    }
};
// the columns (j, j + 4), j = 0 .. 3, of a word as fp16 pairs
__device__ __forceinline__ void w4_unpack(uint32_t w, const W4Const& k, uint32_t (&pair)[4]) {
    const uint32_t v = w >> 8;
    pair[0] = w4_hsub(w4_and_xor<0x000f000fu>(w, k.low), k.low);                // - 1032
    pair[1] = w4_hfma(w4_and_xor<0x00f000f0u>(w, k.high), k.part, k.less);      // / 16 - 72
    pair[2] = w4_hsub(w4_and_xor<0x000f000fu>(v, k.low), k.low);
    pair[3] = w4_hfma(w4_and_xor<0x00f000f0u>(v, k.high), k.part, k.less);
}

// two fp32 values to an fp16 pair, the first in the low half
__device__ __forceinline__ uint32_t w4_pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// all threads of the cluster's CTAs; what they wrote to shared memory is visible to all behind it
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the value at p's place in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// act(g) * u
__device__ __forceinline__ float w4_glu(int act, float g, float u) {
    if (act == DEC_ACT_GELU_TANH) {
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
        const float z = 0.79788456080286536f * fmaf(0.044715f * g * g, g, g);
        return g / (1.0f + expf(-2.0f * z)) * u;
    }
    return g / (1.0f + expf(-g)) * u;
}

// four consecutive values of a row of fp32 or bf16 (16- or 8-byte aligned)
__device__ __forceinline__ float4 w4_load4(const void* p, bool f32, size_t i) {
    if (f32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p) + i);
    return make_float4(bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y));
}
__device__ __forceinline__ float w4_load1(const void* p, bool f32, size_t i) {
    return f32 ? reinterpret_cast<const float*>(p)[i] : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void w4_store1(void* p, bool f32, size_t i, float v) {
    if (f32) reinterpret_cast<float*>(p)[i] = v;
    else reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Activations enter the products as fp16 parts of v * 2^(14 - e), 2^e the power of
// two at or below the largest finite |v| of their block: the scaled values lie
// below 2^15, one part keeps 11 bits of each and two keep 22 (or 2^-39 of the
// block's largest, where that is coarser).  `top` is the largest |v|'s bits.
// fp32 activations have 24 bits: a third part would be half as many products again for
// errors that are below an fp32 product's already (of the whole, against 64 bits, and
// in parentheses the plain fp32 form's: one token 6144 x 4096 1.1e-7 (1.9e-7), eight
// tokens 14336 -> 4096 1.0e-7 (4.2e-7), 1000 tokens gate/up 14336 x 4096 5.6e-7 (1.3e-6)).
__device__ __forceinline__ int w4_exponent(uint32_t top) { return min(max((int)(top >> 23), 15), 254); }
__device__ __forceinline__ float w4_up(int e) { return __uint_as_float((uint32_t)(268 - e) << 23); }     // 2^(14 - (e - 127))
__device__ __forceinline__ float w4_down(int e) { return __uint_as_float((uint32_t)(e - 14) << 23); }    // its reciprocal
__device__ __forceinline__ uint32_t w4_finite_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// the fp16 pair of two scaled values, and that of what it leaves (0 where not finite)
__device__ __forceinline__ uint32_t w4_rest(float a, float b, uint32_t hi) {
    const __half2 h = *reinterpret_cast<const __half2*>(&hi);
    const float ra = a - __low2float(h), rb = b - __high2float(h);
    return w4_pack_half(isfinite(ra) ? ra : 0.f, isfinite(rb) ? rb : 0.f);
}

}  // namespace gd
