// The 8-bit KV cache: what its codes stand for, shared by the kernels that write
// it, read it back and attend over it.
//
// value = code * scale, one float32 scale for every kKv8Block slots of a
// (sequence, head), K and V apart; code int8 in [-127, 127] or e4m3 (finite).
// The write kernel's scales are powers of two: x / scale and code * scale are
// exact, so the code's own rounding is the only one, every code * scale is a
// bf16 number (at most 8 significant bits), and a block whose scale grows
// while it fills is rounded again by a plain shift of its codes' binary point.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace bloom {

constexpr int kKv8Block = 32;   // slots per scale (BLOOM_KV8_BLOCK)

// Four int8 codes of a word -> 4 floats: each byte code + 128 as the last bits of
// 2^23 + byte, less 2^23 + 128 (exact, and no conversion instruction).
__device__ __forceinline__ void kv8_widen_s8(uint32_t w, float *f) {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u + i)) - 8388736.f;
}
// Two floats -> bf16x2, rounded half to even.
__device__ __forceinline__ uint32_t kv8_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes -> f16x2 (exact: 4 significant bits, exponents -9 .. 8).
__device__ __forceinline__ uint32_t kv8_e4m3x2_f16x2(uint16_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return r;
}
__device__ __forceinline__ float kv8_f16lo(uint32_t v) {
    float f;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(v));
    return f;
}
__device__ __forceinline__ float kv8_f16hi(uint32_t v) {
    float f;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, h;\n}\n" : "=f"(f) : "r"(v));
    return f;
}
__device__ __forceinline__ void kv8_widen_e4m3(uint32_t w, float *f) {
    const uint32_t a = kv8_e4m3x2_f16x2((uint16_t)w), b = kv8_e4m3x2_f16x2((uint16_t)(w >> 16));
    f[0] = kv8_f16lo(a);
    f[1] = kv8_f16hi(a);
    f[2] = kv8_f16lo(b);
    f[3] = kv8_f16hi(b);
}
template <bool E4M3>
__device__ __forceinline__ void kv8_widen(uint32_t w, float *f) {
    if (E4M3) kv8_widen_e4m3(w, f);
    else kv8_widen_s8(w, f);
}

// Four floats (already divided by the scale) -> four codes, round half to even.
template <bool E4M3>
__device__ __forceinline__ uint32_t kv8_narrow(float a, float b, float c, float d) {
    uint32_t r;
    if (E4M3) {
        asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
            " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    } else {
        uint32_t hi;
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;"
            : "=r"(hi)
            : "r"(__float2int_rn(d)), "r"(__float2int_rn(c)));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
            : "=r"(r)
            : "r"(__float2int_rn(b)), "r"(__float2int_rn(a)), "r"(hi));
    }
    return r;
}

// Scale of a block whose largest magnitude has the bf16 bits `amax` (sign 0):
// the smallest power of two, 2^-126 at least, with amax <= 127 * scale (int8,
// 127 = 1.984375 * 2^6) or 448 * scale (e4m3, 448 = 1.75 * 2^8); 0 for 0, NaN
// for an infinity or NaN.
template <bool E4M3>
__device__ __forceinline__ float kv8_scale(uint32_t amax) {
    if (amax == 0) return 0.f;
    if (amax >= 0x7f80u) return __uint_as_float(0x7fc00000u);
    const int exp = (int)(amax >> 7), frac = (int)(amax & 127u);   // biased exponent, fraction * 128
    const int e = E4M3 ? exp - 8 + (frac > 96) : exp - 6 + (frac > 126);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

}  // namespace bloom
