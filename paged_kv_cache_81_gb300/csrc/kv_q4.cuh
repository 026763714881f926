// Rows held in 4 bits: groups of 16 elements of a head, each with one e4m3 scale; codes are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives), so an element takes 4.5 bits.  A code times its scale has at most six significant bits: fp16 holds
// it exactly.
//
// A row of `heads` heads of `dim` elements: heads * dim / 2 bytes of codes (element 2 i in the low half of byte i), then
// heads * dim / 16 scales in the same order, filled up to a multiple of 16 bytes.  Codes and scales apart keep every
// head's codes on a 16-byte boundary, and the rows opaque to the calls that move them.
#pragma once

#include <cstdint>

#include "kv_common.cuh"

namespace pkv {

constexpr int kQ4MaxDim = 128;  // of a head; a multiple of 32

inline int64_t q4_row_bytes(int64_t heads, int64_t dim) { return (heads * dim * 9 + 255) / 256 * 16; }

// One plane of one tensor as 4-bit rows.
int check_q4_plane(const kv_cache_desc *c, int tensor, int plane, int heads, int dim);

// The eight values of a word of codes, in order, as pairs of fp16.
__device__ __forceinline__ void q4_to_f16(uint32_t w, uint32_t (&v)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
}

// Eight values as codes, each rounded to the nearest (ties to the even code), in order.
__device__ __forceinline__ uint32_t f32_to_q4(const float (&z)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    return w;
}

// Two scales (bytes of the low half of `b`) as fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t b)
{
    uint32_t v;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"((uint16_t)b));
    return v;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t v;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(a), "r"(b));
    return v;
}

// The scale byte of a group whose largest magnitude is `most`: the nearest e4m3 to most / 6, at most 448 and at least
// 2^-9 (so that no scale is 0).
__device__ __forceinline__ uint32_t q4_scale_of(float most)
{
    uint16_t b;
    asm("{\n\t.reg .f32 z;\n\tmov.f32 z, 0f00000000;\n\tcvt.rn.satfinite.e4m3x2.f32 %0, z, %1;\n\t}" : "=h"(b) : "f"(__fdiv_rn(most, 6.0f)));
    return max((uint32_t)(b & 0xffu), 1u);
}

}  // namespace pkv
