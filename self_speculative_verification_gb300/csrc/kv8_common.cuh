// The 8-bit KV cache: its layout, e4m3 conversions, and the exponent of a
// block's scale.
#pragma once

#include "common.cuh"

namespace sv {
namespace {

constexpr int kKv8MinExp = -60, kKv8MaxExp = 60;
constexpr int kKv8MaxPage = 256;

// First byte of a (page, head) block's tile, and the byte of token t's key
// (x = 0) or value (x = 1) row within it: [page_size / 8][2][8][d].
__device__ __forceinline__ size_t kv8_block(int page, int h, int Hkv, int ps, int d) {
    return ((size_t)page * Hkv + h) * (size_t)(2 * ps * d);
}
__device__ __forceinline__ int kv8_row(int t, int x, int d) {
    return (((t >> 3) * 2 + x) * 8 + (t & 7)) * d;
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A reader's scale: finite ones lie in [2^-60, 2^60]; NaN stays NaN.
__device__ __forceinline__ float kv8_read_scale(float s) {
    if (s != s) return s;
    return fminf(fmaxf(s, exp2_int(kKv8MinExp)), exp2_int(kKv8MaxExp));
}

// Smallest e with a <= 448 * 2^e (a >= 0, finite), within [-60, 60]:
// 448 = 1.75 * 2^8, so it is a's exponent - 8, one more past 1.75.
__device__ __forceinline__ int kv8_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kKv8MinExp), kKv8MaxExp);
}

// Two values as e4m3 (nearest even, saturating; NaN stays NaN): lo in the
// low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low 16 bits) as fp32: every e4m3 value is a half.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

}  // namespace
}  // namespace sv
