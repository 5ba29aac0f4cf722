// qc_mx.hpp -- device-side building blocks of MXFP4: groups of 32 E2M1 values
// with a power-of-two scale.
#pragma once
#include "qc_matrix.hpp"

namespace qc {

constexpr int kMxGroup = 32;
constexpr uint32_t kMxNaN = 255u;

// The scale byte E + 127 of a group whose largest magnitude has these bits: E
// is the smallest integer with amax < 7 * 2^E.  7 = 1.75 * 2^2, so E is amax's
// own exponent less 2, plus one where its fraction is 1.75 or more (the
// addition carries into the exponent field exactly then).  Within [1, 253]: the
// scale and its reciprocal are normal numbers.
__device__ __forceinline__ uint32_t mx_byte(uint32_t amax_bits) {
    const int e = (int)((amax_bits + 0x200000u) >> 23) - 2;
    return amax_bits >= kInfBits ? kMxNaN : (uint32_t)min(max(e, 1), 253);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Codes of eight values of a group: the conversion divides by the power of two
// exactly, rounds to nearest even and keeps signs (of zeros too).
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float scale) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    return w;
}

// The scale as a number (byte 255: only asked for with its codes dropped).
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace qc
