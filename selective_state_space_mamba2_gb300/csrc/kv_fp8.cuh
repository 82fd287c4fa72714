// A cache in 8 bits: e4m3 codes and a scale for each block and key head (device helpers).
#pragma once
#include "kv.cuh"

namespace ssd {
namespace fp8 {

constexpr int kLeast = -64, kMost = 119;  // exponents of the scales that are written: code * scale is a normal, finite float

// Codes of a (low byte) and b, rounded to nearest even; beyond 448: 448; NaN stays NaN.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Values of the two codes in the low half of v.
__device__ __forceinline__ float2 decode2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ void decode8(uint2 c, float (&v)[8]) {
    const float2 a = decode2(c.x), b = decode2(c.x >> 16), d = decode2(c.y), e = decode2(c.y >> 16);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = d.x, v[5] = d.y, v[6] = e.x, v[7] = e.y;
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8]) {
    return make_uint2(encode2(v[0], v[1]) | encode2(v[2], v[3]) << 16, encode2(v[4], v[5]) | encode2(v[6], v[7]) << 16);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The smallest power of two s with top <= 448 s (448 = 1.75 * 2^8), within the limits; top finite, not negative.
__device__ __forceinline__ float scale_for(float top) {
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
    return __uint_as_float((uint32_t)(min(max(e, kLeast), kMost) + 127) << 23);
}

// Where r of the S ascending values base(0) <= base(1) ... is the last that is at most `x`; called by whole warps.
// (values that do not ascend give some r in [0, S))
template <typename F> __device__ __forceinline__ int last_at_most(int S, long long x, F base) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const uint32_t yes = __ballot_sync(~0u, at < hi && base(at) <= x);
        lo += yes ? (31 - __clz(yes)) * step : 0;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace fp8
}  // namespace ssd
