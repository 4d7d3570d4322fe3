// The 4-bit row format (OXD_FORMAT_E2M1 in oxd.h): groups of 32 columns with
// one f16 scale and 32 e2m1 codes. Shared by the append, the page copies and
// the decode.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "oxd_internal.h"

namespace oxd {
namespace {

constexpr int kScaleGroup = 32;           // columns that share a scale
constexpr int kRowScales = kHeadDim / kScaleGroup;
// The largest scale: six times it is the largest value held, 65472, below the
// largest f16, so code x scale never overflows where it is formed in f16.
constexpr float kMaxScale = 10912.f;

// f16 scale bits of a group whose largest size is `amax` (a bf16 value): the
// f16 number nearest to amax / 6. The f32 quotient rounds to the same f16
// number as the exact one: amax has 8 significant bits, so amax / 6 either has
// no more (a multiple of 3) or repeats in binary and stays clear of the
// midpoints of 11-bit numbers by far more than f32 rounds.
__device__ __forceinline__ uint16_t group_scale(float amax) {
    return __half_as_ushort(__float2half_rn(fminf(__fdiv_rn(amax, 6.f), kMaxScale)));
}

// 1 / scale for code_pair; 0 for a group of zeros.
__device__ __forceinline__ float scale_inverse(uint16_t scale) {
    const float s = __half2float(__ushort_as_half(scale));
    return s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
}

// Codes of two neighbouring columns (x0 in the low half of the byte), each the
// e2m1 number nearest to x / s, ties to even. inv = 1 / s rounded, so x * inv
// may miss a quotient that lies exactly between two codes by a rounding; the
// quotient of an 8-bit by an 11-bit number that is no tie differs from one by
// at least 2^-16 (a tie is at least 0.25 and t * s has 14 bits), so rounding
// x * inv to a multiple of 2^-17, by adding and taking away 1.5 * 2^6, restores
// ties and moves nothing across one.
__device__ __forceinline__ uint32_t code_pair(float x0, float x1, float inv) {
    constexpr float kGrid = 96.f;
    const float y0 = __fadd_rn(fmaf(x0, inv, kGrid), -kGrid);
    const float y1 = __fadd_rn(fmaf(x1, inv, kGrid), -kGrid);
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "mov.b32 %0, {b, 0, 0, 0};\n\t}"
        : "=r"(r)
        : "f"(y1), "f"(y0));
    return r;
}

// The four code pairs of a 32-bit word as f16x2 (low half: the even column).
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Byte offset of the codes of (page, token t, head h), and index of the row's
// first scale.
__device__ __forceinline__ size_t row_index(int layout, int64_t page, int t, int h, int H, int ps) {
    return layout == 0 ? (static_cast<size_t>(page) * ps + t) * H + h
                       : (static_cast<size_t>(page) * H + h) * ps + t;
}
__device__ __forceinline__ size_t scale_index(int64_t page, int t, int h, int H, int ps) {
    return ((static_cast<size_t>(page) * H + h) * ps + t) * kRowScales;
}

}  // namespace
}  // namespace oxd
