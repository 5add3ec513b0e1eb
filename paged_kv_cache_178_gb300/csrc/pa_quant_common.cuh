// 4-bit cache records and the conversions between codes, scales and values,
// shared by the write, the read-back and the attention.
//
// For one page and KV head, K and V each have a record of 9*DH bytes:
//   K: codes [16 tokens][DH/2], then scales [16 tokens][DH/16];
//   V: codes [DH/2][16 tokens], then scales [DH/16][16 tokens].
// A code byte holds the e2m1 codes of two neighbouring head-dim elements of a
// token (the even one in the low half), a scale byte the e4m3 factor of 16
// neighbouring elements.  K is token-major because its attention product
// reduces over the head dim, V is head-dim-major because its product reduces
// over the tokens: either way one 32-bit load brings four of the bytes a
// matrix fragment needs.
#pragma once
#include <cstdint>

namespace pa {

__host__ __device__ constexpr int quant_record_bytes(int dh) { return 9 * dh; }
__host__ __device__ constexpr int quant_code_bytes(int dh) { return 8 * dh; }

// Eight codes -> four f16 pairs (exact): pair i is byte i, low half first.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Two scale bytes (in the low half of w) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w)
{
    uint32_t o;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(o)
        : "r"(w));
    return o;
}

// Products of an f16 code pair and an f16 scale pair: exact (two significant
// bits times four; the smallest, 2^-10, is a normal f16, the largest 2688).
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t o;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}

}  // namespace pa
