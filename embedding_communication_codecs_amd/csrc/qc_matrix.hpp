// qc_matrix.hpp -- device-side building blocks of the matrix operators
// (INT8 rows, 8-bit checkpoints and the products over them).
#pragma once
#include "qc_device.hpp"

namespace qc {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 bytes at any element alignment: rows of a matrix whose row stride is
// odd start at odd elements, and gfx950 loads and stores those in one
// instruction too.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

struct BF16 {  // storage of one bf16 value
    uint16_t b;
};

__device__ __forceinline__ float to_f32(BF16 x) { return bf16_to_f32(x.b); }
__device__ __forceinline__ float to_f32(float x) { return x; }

// fp32 to bf16, to nearest even (v_cvt_pk_bf16_f32; a NaN stays a NaN).
__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ void put(BF16* p, float v) { p->b = bf16_bits(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// The first `left` of eight consecutive values, fewer than eight, the rest +0.
// Loads of neighbours stand in for those past the end, so that all are on
// their way at a time (INT8 rows of 15012 x 6733 bf16: 72 us against 84
// with a load and a branch each).
template <class T>
__device__ __forceinline__ void load_some(const T* p, int64_t left, float (&v)[8]) {
    const int have = left > 0 ? (int)left : 0;
    T raw[8] = {};
    if (have > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = p[min(i, have - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < have ? to_f32(raw[i]) : 0.0f;
}

// Eight consecutive values; only the first `left` exist (the rest read as +0).
__device__ __forceinline__ void load8(const BF16* p, int64_t left, float (&v)[8]) {
    if (left >= 8) {
        const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        load_some(p, left, v);
    }
}
__device__ __forceinline__ void load8(const float* p, int64_t left, float (&v)[8]) {
    if (left >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p + 4 * h));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(w[i]);
        }
    } else {
        load_some(p, left, v);
    }
}
__device__ __forceinline__ void store8(BF16* p, int64_t left, const float (&v)[8]) {
    if (left >= 8) {
        const u32x4 w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) put(p + i, v[i]);
    }
}
__device__ __forceinline__ void store8(float* p, int64_t left, const float (&v)[8]) {
    if (left >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * h + i]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(p + 4 * h));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = v[i];
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// 1.5 * 2^23: a number of magnitude up to 2^22 added to it is rounded to a
// whole number, to nearest even, whose two's complement low bits are those
// of the sum's bit pattern.
constexpr float kWhole = 12582912.0f;

// The low bytes of four such sums as a word, the first lowest.
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000C0Cu);
    return lo | hi;
}

constexpr uint32_t kInfBits = 0x7F800000u;

// ------------------------------------------------------- checkpoint steps
// The step of a group of 32 values is 2^E, E the smallest integer with
// amax <= 127 * 2^E, held as the byte E + 127.  127 = 1.984375 * 2^6, so E
// is amax's own exponent less 6, plus one where its mantissa exceeds that
// of 1.984375 (the addition below carries into the exponent field exactly
// then).  The byte stays within [1, 248]: the step and its reciprocal are
// normal numbers and 127 steps stay finite.  255 marks a group that holds
// an infinity or a NaN: its step reads as infinity and its codes are 0,
// whose product is NaN.
constexpr uint32_t kCkptNaN = 255u;
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax_bits) {
    const int e = (int)((amax_bits + 0x1FFFFu) >> 23) - 6;
    return amax_bits >= kInfBits ? kCkptNaN : (uint32_t)min(max(e, 1), 248);
}
__device__ __forceinline__ float ckpt_step(uint32_t byte) { return __uint_as_float(byte << 23); }
// Codes of eight values of a group with exponent byte `byte`.  The
// multiply-add rounds the exact x * 2^-E once, to a whole number; a byte of
// 248 may stand for a group beyond 127 steps.
__device__ __forceinline__ u32x2 ckpt_codes(const float (&v)[8], uint32_t byte) {
    const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
    const float most = 127.0f * ckpt_step(min(byte, 248u));
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(fminf(fmaxf(v[i], -most), most), inv, kWhole);
    const bool nan = byte == kCkptNaN;
    return u32x2{nan ? 0u : low_bytes(s[0], s[1], s[2], s[3]), nan ? 0u : low_bytes(s[4], s[5], s[6], s[7])};
}

// Byte i of a word as a signed code (one conversion instruction).
__device__ __forceinline__ float code_of(uint32_t word, int i) { return (float)(int8_t)(word >> (8 * i)); }

// Eight codes times their step, exactly.  A step of infinity (byte 255) with
// its codes 0 gives NaN.
__device__ __forceinline__ void ckpt_values(u32x2 codes, uint32_t byte, float (&v)[8]) {
    const float step = ckpt_step(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = code_of(codes[i >> 2], i & 3) * step;
}

// Maximum over aligned groups of four lanes (8 values each: one group).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) { return group_max_u32<4>(v); }

}  // namespace qc
