// row_codes.cuh -- the codes of a latent cache row widened to fp16, and the fp16 helpers of the
// attention kernels that read such rows.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace glm {

// Four int8 codes (one little-endian word) as four exact fp16 values (two fp16x2 words).
__device__ __forceinline__ void codes_to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t t = w ^ 0x80808080u;                          // each code c as the byte c + 128
    const uint32_t a = __byte_perm(t, 0x64646464u, 0x5140u);     // fp16 bits 0x64bb = 1024 + c + 128
    const uint32_t b = __byte_perm(t, 0x64646464u, 0x5342u);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));   // - 1152 (exact)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}
// Eight E2M1 codes (one word, low nibble first) as eight fp16 values times the fp16 block scale
// sc2 (in both halves): exact, since a 2-bit by 4-bit significand product of magnitude in
// [2^-10, 2688] is an fp16 normal.
__device__ __forceinline__ void fp4_to_f16x8(uint32_t w, uint32_t sc2, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; i++) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(sc2));
}
// Four E4M3 codes as four exact fp16 values (hardware conversion of code pairs).
__device__ __forceinline__ void fp8_to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    lo = static_cast<uint32_t>(a.x) | (static_cast<uint32_t>(a.y) << 16);
    hi = static_cast<uint32_t>(b.x) | (static_cast<uint32_t>(b.y) << 16);
}

__device__ __forceinline__ uint32_t f16x2_rn(float a, float b) {   // .x = a (low half)
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float f16_lo_f(uint32_t p) { return __half2float(__ushort_as_half(static_cast<unsigned short>(p & 0xffffu))); }
__device__ __forceinline__ float f16_hi_f(uint32_t p) { return __half2float(__ushort_as_half(static_cast<unsigned short>(p >> 16))); }

// The smallest power of two >= x (1 for x <= 0, capped at 2^127).
__device__ __forceinline__ float pow2_ceil(float x) {
    if (!(x > 0.0f)) return 1.0f;
    const uint32_t b = __float_as_uint(x);
    int e = static_cast<int>(b >> 23) - 127;
    if ((b & 0x7fffffu) != 0u || e < -126) e += 1;
    e = max(-126, min(127, e));
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace glm
