// kv8.cuh -- what the kernels of the 8-bit K/V cache share: the launch
// parameters, which tokens and positions a row has, where a position lies, and
// the conversions between e4m3 and wider types.
//
// A stored value is x8 * 2^e: x8 in e4m3 (1 sign, 4 exponent, 3 mantissa bits,
// no infinity) and one exponent e, held as the byte e + 127, for each block of
// `block` consecutive positions of one K/V head.  A power of two changes no
// significant bit, so e4m3 and 2^e multiply without rounding anywhere.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "common.cuh"
#include "internal.h"

namespace gd {

constexpr float KV8_LOG2E = 1.4426950408889634f;

// ---- rows ----
struct Kv8Row {
    int t0, n;   // its packed tokens [t0, t0 + n)
    int len;     // positions of the row after those tokens: token i is position len - n + i
};
// false: the row's entries are out of range (FAULT_POS); nothing of it is touched
__device__ __forceinline__ bool kv8_row(const Kv8Batch& b, int cap, int r, Kv8Row* out) {
    if (!b.kv_len) {   // one row, by the launch
        *out = Kv8Row{0, b.total, b.len_add};
        return true;
    }
    const int t0 = b.q_start ? b.q_start[r] : r;
    const int t1 = b.q_start ? b.q_start[r + 1] : r + 1;
    const int len = (int)((unsigned)b.kv_len[r] + (unsigned)b.len_add);
    if (t0 < 0 || t1 < t0 || t1 > b.total || t1 - t0 > b.max_new || len < 0 || len > cap) {
        atomicOr(b.err, FAULT_POS);
        return false;
    }
    *out = Kv8Row{t0, t1 - t0, len};
    return true;
}
// the page that holds page slot i of row r, or -1 (FAULT_SLOT_MAP) if its id is out of range
__device__ __forceinline__ int kv8_page(const Kv8Cache& c, unsigned* err, int r, int i) {
    const int id = c.pages ? c.pages[(size_t)r * c.ppr + i] : r * c.ppr + i;
    if ((unsigned)id >= (unsigned)c.num_pages) {
        atomicOr(err, FAULT_SLOT_MAP);
        return -1;
    }
    return id;
}
// whether a token at position p sees position j; `window` is INT_MAX without one
__device__ __forceinline__ bool kv8_sees(int p, int j, int window, int sinks) {
    return j <= p && (j > p - window || j < sinks);
}

// ---- e4m3 ----
// two e4m3 values (low and high byte) of each half of w as packed f16 pairs; exact, NaN stays NaN
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    e4m3x4_to_f16(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
// four fp32 values (|x| <= 448, or NaN) to e4m3, round to nearest even
__device__ __forceinline__ uint32_t f32_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n"
        " mov.b32 %0, {x, y};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
constexpr int KV8_EXP_MIN = -40, KV8_EXP_MAX = 60;

// least e with top <= 448 * 2^e; 448 = 1.75 * 2^8
__device__ __forceinline__ int kv8_exponent(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, KV8_EXP_MIN), KV8_EXP_MAX);
}

// scale bytes with which attention's sums stay in fp32's range (2^-100 .. 2^100); others are flagged (FAULT_SCALE)
__device__ __forceinline__ bool kv8_scale_ok(int byte) { return (unsigned)(byte - 27) <= 200u; }

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// 2^x by the hardware's base-2 exponential
__device__ __forceinline__ float kv8_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace gd
