// qx_attn_codes.cuh -- the codes of an 8-bit cache as the tensor cores take them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace qx {

// Four codes as two pairs of f16: the bytes LO and HI of c + 128 in the low byte
// of 0x6400 (1024, where f16 counts by ones), less 1152.
template <int LO, int HI>
__device__ __forceinline__ uint32_t code_pair(uint32_t biased) {
    const uint32_t u = __byte_perm(biased, 0x64646464u, LO | 0x40 | HI << 8 | 0x4000);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The same as bf16, which counts by ones from 128 to 255 only: 128 and the low seven
// bits, less 128, or 256 where the code is negative.
template <int LO, int HI>
__device__ __forceinline__ uint32_t code_pair_bf16(uint32_t codes) {
    const uint32_t u = __byte_perm(codes, 0x43434343u, LO | 0x40 | HI << 8 | 0x4000);
    const uint32_t low = u & 0xff7fff7fu, less = u & 0xff80ff80u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&low), *reinterpret_cast<const __nv_bfloat162*>(&less));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float power_of_two(int exponent_field) { return __uint_as_float(uint32_t(exponent_field) << 23); }

// A row's probabilities are multiplied by its values' scales before they are
// rounded, so its running base is the largest score plus the least power of two
// that no scale reaches (from 2^-80 on): so much are the probabilities and their
// sum raised, and the products stay below the base's 1.  The base may be 80 powers
// below the row's largest score, where its sum is up to 2^95 a key, or as much
// above it as the scales are large; a sum goes from one base to the other whole
// (twice(), qx_attn.cuh), while products that many powers down are nothing.
// (2^-80: with a power of 2^-100 the sum, of 2^115 a key, would leave f32 at 8192
// keys.  Values whose scales are all below 2^-80 keep what f16 leaves of them.)
constexpr float kLeastPower = -80.0f;
__device__ __forceinline__ float scale_power(float d) {
    return fmaxf(float(int(__float_as_uint(d) >> 23 & 0xff) - 126), kLeastPower);
}

}  // namespace qx
