// Block-scaled storage shared by the sources of libmoe_native (internal):
// groups of 32 columns, one scale byte b = 2^(b - 127) each.
#pragma once

#include "../../include/moe_lowbit.h"
#include "moe_common.h"

namespace moe {
namespace {

constexpr int kGroup = 32;          // columns that share a scale byte
constexpr int kScaleNaN = 255;      // the scale byte of a group that stands for NaN

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale bytes from a group's largest magnitude, as the bits of the float (an
// integer maximum keeps NaN above infinity above every number).  The codes
// reach M = 127 (q8) or 6 (w4); the exponent of amax less the power of two in
// M is the scale, one more where amax would round past M: from 127.5 = 1.9921875
// * 2^6, or 7 = 1.75 * 2^2, on.  Adding the distance of that mantissa from 2
// carries exactly those into the exponent.  An exponent of 255 then is a NaN,
// an infinity, or a magnitude that would round to 2^128.
template <uint32_t CARRY, int BELOW>
__device__ __forceinline__ int scale_byte(uint32_t amax) {
    const int e = static_cast<int>((amax + CARRY) >> 23);
    return e >= 255 ? kScaleNaN : max(e - BELOW, 1);
}
__device__ __forceinline__ int q8_scale_byte(uint32_t amax) { return scale_byte<0x10000u, 6>(amax); }
__device__ __forceinline__ int w4_scale_byte(uint32_t amax) { return scale_byte<0x200000u, 2>(amax); }

// 2^(127 - b) for b in [1, 252]: what a value is multiplied by on its way to
// a code (exact); 0 for a NaN group.
__device__ __forceinline__ float inv_scale(int b) {
    return b == kScaleNaN ? 0.0f : __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
}

// rint(v * inv) as the low byte: adding 1.5 * 2^23 leaves the nearest whole
// number (ties to even) in the low mantissa bits, one rounding in the fma.
// (inf and NaN times inv = 0 are NaN, whose low byte is masked by the caller.)
__device__ __forceinline__ uint32_t q8_code(float v, float inv) {
    return __float_as_uint(__builtin_fmaf(v, inv, 12582912.0f));
}

// Four codes as the bytes of a word.
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d, float inv) {
    return __builtin_amdgcn_perm(q8_code(b, inv), q8_code(a, inv), 0x0C0C0400u) |
           __builtin_amdgcn_perm(q8_code(d, inv), q8_code(c, inv), 0x04000C0Cu);
}

// 2^(b - 127) of a scale byte; a NaN for b = 255.  b = 0 (2^-127, written by
// no quantizer here) is a subnormal.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == kScaleNaN ? 0x7FC00000u : b << 23);
}

// The j-th int8 of a word, as float32.
__device__ __forceinline__ float q8_float(uint32_t word, int j) {
    return static_cast<float>(static_cast<int8_t>(word >> (8 * j)));
}

}  // namespace
}  // namespace moe
