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
// f16 number nearest to amax / 6. The product with the f32 nearest to 1/6 is
// within 2^-23 of the quotient, and rounds to the same f16 number: amax has 8
// significant bits, so amax / 6 either has no more (a multiple of 3) or repeats
// in binary, and stays clear of the midpoints of 11-bit numbers by far more.
// Only below f16's normal range can a quotient be a midpoint; it is divided.
__device__ __forceinline__ uint32_t group_scale(float amax) {
    float q = amax * (1.f / 6.f);
    if (q < 6.2e-5f) q = __fdiv_rn(amax, 6.f);
    return __half_as_ushort(__float2half_rn(fminf(q, kMaxScale)));
}

// 1 / scale, to 2^-23; 0 for a group of zeros.
__device__ __forceinline__ float scale_inverse(uint32_t scale) {
    const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale)));
    return s > 0.f ? __fdividef(1.f, s) : 0.f;
}

// x / s for its code, inv = 1 / s: x * inv may miss a quotient that lies exactly
// between two codes by a rounding. The quotient of an 8-bit by an 11-bit number
// that is no tie differs from one by at least 2^-16 (a tie is at least 0.25, and
// tie * s has 14 bits), and x * inv is within 2^-19 of it up to 6, so rounding
// it to a multiple of 2^-17, by adding and taking away 1.5 * 2^6, restores ties
// and moves nothing across one.
// Two at a time, as packed f32 (half the instructions).
__device__ __forceinline__ void code_arguments(float& x, float& y, float inv) {
    constexpr float kGrid = 96.f;
    asm("{\n\t.reg .b64 u, v, g;\n\t"
        "mov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 g, {%3, %3};\n\t"
        "fma.rn.f32x2 u, u, v, g;\n\tmov.b64 g, {%4, %4};\n\t"
        "add.rn.f32x2 u, u, g;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(inv), "f"(kGrid), "f"(-kGrid));
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Codes of eight columns (bf16 pairs): each the e2m1 number nearest to x / s,
// ties to even, the first column in the lowest four bits.
__device__ __forceinline__ uint32_t code_eight(const uint4& x, float inv) {
    float f[8];
    const uint32_t* w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_low(w[i]);
        f[2 * i + 1] = bf16_high(w[i]);
        code_arguments(f[2 * i], f[2 * i + 1], inv);
    }
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight columns of a row in 4 bits, and their group's f16 scale. The group's
// other columns are in the lanes next to this one (a multiple of four and its
// three followers): every lane of the warp calls it.
__device__ __forceinline__ void hold_eight(const uint4& x, uint32_t& code, uint32_t& scale) {
    // (the larger of a number and a NaN is the number, here and in fmaxf)
    uint32_t m = max_bf16x2(max_bf16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                            max_bf16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    scale = group_scale(fmaxf(bf16_low(m), bf16_high(m)));
    code = code_eight(x, scale_inverse(scale));
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

// Index of the row of (page, token t, head h) in a pool of rows (codes or bf16),
// and of the row's first scale.
__device__ __forceinline__ size_t row_index(int layout, int64_t page, int t, int h, int H, int ps) {
    return layout == 0 ? (static_cast<size_t>(page) * ps + t) * H + h
                       : (static_cast<size_t>(page) * H + h) * ps + t;
}
__device__ __forceinline__ size_t scale_index(int64_t page, int t, int h, int H, int ps) {
    return ((static_cast<size_t>(page) * H + h) * ps + t) * kRowScales;
}

}  // namespace
}  // namespace oxd
