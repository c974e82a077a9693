// The 4-bit format of the key-value cache, for the kernels that write and read it.
//
// A block is 32 consecutive channels of one position and head: a scale byte b,
// 2^(b-127), and 32 codes of 4 bits, a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6.
// The scale is the least power of two with max |x| <= 7 * 2^e: 6 is the largest
// element, and clipping what lies above it up to 7 costs less than doubling the
// spacing of the other 31 (rms error of normal blocks 11.2%, against 11.5% where
// the limit is 6 or 8).  b runs from 1 to 252: every value is then finite, and a
// block below 2^-128 is zeros.  A block with an infinity or NaN stands for NaN:
// b = 255, its codes 0.
//
// Scaling by a power of two is exact and the conversion instruction rounds to
// nearest, ties to the even code, so codes are defined bit by bit.
#pragma once

#include "attn_common.h"

namespace gdr {
namespace attn {

constexpr int kMxBlock = 32;   // channels of a block
constexpr int kMxRows = 32;    // positions of a value block (16 bytes of one channel)
constexpr uint32_t kMxMost = 252, kMxNan = 255;  // the largest scale byte, and that of NaN

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
    const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 2;  // one more above a mantissa of 7/4
    return top >= 0x7f800000u ? kMxNan : static_cast<uint32_t>(min(max(e, 1), static_cast<int>(kMxMost)));
}
// What the values are multiplied by before the conversion; 0 for NaN blocks, whose codes are cleared anyway.
__device__ __forceinline__ float mx_inverse(uint32_t b) { return b == kMxNan ? 0.f : __uint_as_float((254u - b) << 23); }
__device__ __forceinline__ float mx_float(uint32_t b) { return __uint_as_float(b << 23); }
// Of byte n (a constant) of a word, in one instruction; the compiler takes two (64
// sequences of 16 .. 4000 tokens, 16 query rows: 41.7 us against 43.5; fp32, 16 .. 8000:
// 95 against 102).
__device__ __forceinline__ float mx_float(uint32_t w, int n) {
    uint32_t r;
    if (n == 0)
        asm("v_lshlrev_b32_sdwa %0, 23, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0" : "=v"(r) : "v"(w));
    else if (n == 1)
        asm("v_lshlrev_b32_sdwa %0, 23, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1" : "=v"(r) : "v"(w));
    else if (n == 2)
        asm("v_lshlrev_b32_sdwa %0, 23, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2" : "=v"(r) : "v"(w));
    else
        asm("v_lshlrev_b32_sdwa %0, 23, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3" : "=v"(r) : "v"(w));
    return __uint_as_float(r);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Codes of a and b in byte SEL of `to`, a in the low half.
template <int SEL> __device__ __forceinline__ uint32_t mx_put(uint32_t to, float a, float b) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(to, a, b, 1.f, SEL);
}

// The 8 codes of a word times 2^e, exactly, as bf16 (scale: 2^e).
__device__ __forceinline__ bf16x8v mx_bf16(uint32_t w, float scale) {
    typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
    const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return __builtin_bit_cast(bf16x8v, make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                  __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)));
}

}  // namespace attn
}  // namespace gdr
