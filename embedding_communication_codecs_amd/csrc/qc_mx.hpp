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
// The scale as a number; of a group of NaNs 1, as its codes are replaced.  The
// conversions look at its exponent alone and take 0, of byte 0, for 2^-127.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float((byte == kMxNaN ? 127u : byte) << 23);
}

// Values as a group's codes are made from them: fp32, or bf16 two a word.  The
// conversions divide by the power of two exactly, round to nearest even, take
// what is above 6 (below 7) for 6 and keep signs, of zeros too.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int AT>
__device__ __forceinline__ uint32_t mx_code_pair(uint32_t word, float lo, float hi, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, lo, hi, scale, AT);
}
template <int AT>
__device__ __forceinline__ uint32_t mx_code_pair(uint32_t word, uint32_t pair, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, pair), scale, AT);
}

// Eight codes; v: values, or words of two.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float scale) {
    uint32_t w = mx_code_pair<0>(0u, v[0], v[1], scale);
    w = mx_code_pair<1>(w, v[2], v[3], scale);
    w = mx_code_pair<2>(w, v[4], v[5], scale);
    return mx_code_pair<3>(w, v[6], v[7], scale);
}
__device__ __forceinline__ uint32_t mx_codes8(u32x4 v, float scale) {
    uint32_t w = mx_code_pair<0>(0u, v[0], scale);
    w = mx_code_pair<1>(w, v[1], scale);
    w = mx_code_pair<2>(w, v[2], scale);
    return mx_code_pair<3>(w, v[3], scale);
}

// The larger magnitudes of two bf16 values a word, m those so far; and the
// largest of both as fp32 bits.
__device__ __forceinline__ uint32_t pair_max(uint32_t m, uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t amax_of_pair(uint32_t m) { return umax(m << 16, m & 0xFFFF0000u); }

// Eight neighbouring values of a row as they lie in memory, zeros where there
// are none.  load() asks for them without a wait: at a row's end for the last
// eight of the row (`back`: there are eight before), which settle() then moves
// to their places, so that lanes at the end of a row cost no load after the
// other (1027 x 770 fp32 in both orientations: 10 us with a wait in each of a
// lane's eight loads).  Rows of fewer than eight are loaded value by value.
template <class T>
struct Raw8;
template <>
struct Raw8<BF16> {
    u32x4 w;
    // m: magnitudes so far, from 0; bits_of(m): the largest as fp32 bits
    __device__ __forceinline__ uint32_t max_with(uint32_t m) const {
        return pair_max(pair_max(pair_max(pair_max(m, w[0]), w[1]), w[2]), w[3]);
    }
    __device__ __forceinline__ static uint32_t bits_of(uint32_t m) { return amax_of_pair(m); }
    __device__ __forceinline__ uint32_t amax_bits() const { return bits_of(max_with(0u)); }
    __device__ __forceinline__ uint32_t codes(float scale) const { return mx_codes8(w, scale); }
    template <bool STREAM>
    __device__ __forceinline__ void load(const BF16* p, int64_t left, bool back) {
        w = u32x4{0, 0, 0, 0};
        if (left >= 8 || (left > 0 && back)) {
            const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(left >= 8 ? p : p + left - 8);
            w = STREAM ? (u32x4)__builtin_nontemporal_load(q) : (u32x4)*q;
        } else if (left > 0) {
            float v[8];
            load_some(p, left, v);
            w = u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
        }
    }
    __device__ __forceinline__ void settle(int64_t left, bool back) {
        if (left > 0 && left < 8 && back) {
            const int by = 8 - (int)left;
            if (by & 4) w = u32x4{w[2], w[3], 0, 0};
            if (by & 2) w = u32x4{w[1], w[2], w[3], 0};
            if (by & 1)
                w = u32x4{(w[0] >> 16) | (w[1] << 16), (w[1] >> 16) | (w[2] << 16), (w[2] >> 16) | (w[3] << 16),
                          w[3] >> 16};
        }
    }
};
template <>
struct Raw8<float> {
    float v[8];
    __device__ __forceinline__ uint32_t max_with(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(v[i]));
        return m;
    }
    __device__ __forceinline__ static uint32_t bits_of(uint32_t m) { return m; }
    __device__ __forceinline__ uint32_t amax_bits() const { return max_with(0u); }
    __device__ __forceinline__ uint32_t codes(float scale) const { return mx_codes8(v, scale); }
    template <bool STREAM>
    __device__ __forceinline__ void load(const float* p, int64_t left, bool back) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (left >= 8 || (left > 0 && back)) {
            const float* from = left >= 8 ? p : p + left - 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(from + 4 * h);
                const u32x4 w = STREAM ? (u32x4)__builtin_nontemporal_load(q) : (u32x4)*q;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(w[i]);
            }
        } else if (left > 0) {
            load_some(p, left, v);
        }
    }
    __device__ __forceinline__ void settle(int64_t left, bool back) {
        if (left > 0 && left < 8 && back) {
#pragma unroll
            for (int by = 4; by >= 1; by >>= 1) {
                if ((8 - (int)left) & by) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = i + by < 8 ? v[i + by] : 0.0f;
                }
            }
        }
    }
};

}  // namespace qc
