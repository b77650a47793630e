// fp4.cuh — the 4-bit K/V cache: its layout and conversions.
//
// A row is one (token, kv head): 128 numbers as 64 bytes of E2M1 codes (two
// to a byte, the even channel in the low half) and 8 bytes of E4M3 group
// scales, one per 16 channels. A number is layer_scale * E4M3(scale) *
// E2M1(code). E2M1 (1 sign, 2 exponent bits with bias 1, 1 mantissa bit) holds
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; E4M3 has 4 significant
// bits, so the product of the two has at most 6 and lies in [2^-10, 2688]:
// an fp16 and a bf16 exactly.
#pragma once

#include "common.cuh"

namespace lsa {

constexpr int kFp4D = 128;                       // channels of a row
constexpr int kFp4Group = 16;                    // channels that share a scale
constexpr int kFp4CodeBytes = kFp4D / 2;         // 64
constexpr int kFp4Groups = kFp4D / kFp4Group;    // 8 scale bytes
constexpr uint32_t kE4m3NaN = 0x7fu;

// Four bytes of two codes each -> four fp16 pairs (low code in the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 c0, c1, c2, c3;\n mov.b32 {c0, c1, c2, c3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, c0;\n cvt.rn.f16x2.e2m1x2 %1, c1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c2;\n cvt.rn.f16x2.e2m1x2 %3, c3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// Eight numbers -> eight codes, x[0] in the lowest four bits; to nearest,
// ties to the even code, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n .reg .b8 c0, c1, c2, c3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n"
        " mov.b32 %0, {c0, c1, c2, c3};\n}\n"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Two E4M3 bytes (low first) -> an fp16 pair (NaN stays NaN).
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint16_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
    return *reinterpret_cast<const __half2*>(&r);
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
    return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace lsa
