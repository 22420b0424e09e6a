// The numbers that a quantized cache's codes stand for: the fp16 number nearest
// to scale * code + bias, one rounding for each.
//
// A code in a half's low bits below the exponent of 1024 is 1024 + code exactly;
// a packed subtraction leaves the code, a packed multiply-add rounds once. Codes
// come out in the head's order: bytes are put beside the exponent byte by a byte
// permutation, after 4-bit codes were spread over bytes.
#pragma once

#include "qmm_device.hpp"

namespace qmm {

// Four bytes of `bytes`, which are codes, as numbers.
__device__ __forceinline__ u32x2 code_numbers(uint32_t bytes, half2_t scale, half2_t bias)
{
    const half2_t magic = {(_Float16)1024.0f, (_Float16)1024.0f};
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // bytes 2i and 2i + 1 under 0x64
        const uint32_t w = __builtin_amdgcn_perm(0x64646464u, bytes, i == 0 ? 0x04010400u : 0x04030402u);
        const half2_t c = __builtin_bit_cast(half2_t, w) - magic;
        r[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, scale, bias));
    }
    return r;
}

// 8 codes (u32x2 of 8-bit codes, one word of 4-bit codes) with their
// (scale, bias) word.
template <int BITS>
struct Eight;
template <>
struct Eight<8> {
    typedef u32x2 raw;
};
template <>
struct Eight<4> {
    typedef uint32_t raw;
};
__device__ __forceinline__ u32x4 eight_numbers(uint32_t low, uint32_t high, uint32_t sb)
{
    const half2_t both = __builtin_bit_cast(half2_t, sb);
    const half2_t s = {both.x, both.x}, b = {both.y, both.y};
    const u32x2 x = code_numbers(low, s, b), y = code_numbers(high, s, b);
    return u32x4{x.x, x.y, y.x, y.y};
}
__device__ __forceinline__ u32x4 eight_numbers(u32x2 codes, uint32_t sb) { return eight_numbers(codes.x, codes.y, sb); }
__device__ __forceinline__ u32x4 eight_numbers(uint32_t codes, uint32_t sb)
{
    const uint32_t even = codes & 0x0F0F0F0Fu, odd = codes >> 4 & 0x0F0F0F0Fu;
    return eight_numbers(__builtin_amdgcn_perm(odd, even, 0x05010400u), __builtin_amdgcn_perm(odd, even, 0x07030602u), sb);
}

// Eight 4-bit codes in the order 0, 2, 4, 6, 1, 3, 5, 7, which takes 11 operations
// instead of 17: a byte of 0 .. 15 is that many steps of 2^-9 as an e4m3 number (the
// subnormal ones and the first binade), so a conversion forms two codes.
__device__ __forceinline__ u32x4 eight_paired_numbers(uint32_t codes, uint32_t sb)
{
    const half2_t both = __builtin_bit_cast(half2_t, sb);
    const half2_t s = {both.x, both.x}, b = {both.y, both.y};
    const uint32_t even = codes & 0x0F0F0F0Fu, odd = codes >> 4 & 0x0F0F0F0Fu;
    auto two = [&](auto c) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, c), s, b));
    };
    return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 0x1p9f, false)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 0x1p9f, true)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 0x1p9f, false)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 0x1p9f, true))};
}
// Eight 16-bit values in that order.
__device__ __forceinline__ u32x4 paired(u32x4 v)
{
    return u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                 __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
}

}  // namespace qmm
