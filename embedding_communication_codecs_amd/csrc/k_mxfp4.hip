// k_mxfp4.hip -- matrices to MXFP4 and back: codes and scale bytes of a matrix
// and of its transpose.
#include "qc_launch.hpp"
#include "qc_mx.hpp"

namespace qc {
namespace {

// Thread (row, group): 32 values of a row, `step` elements apart.
template <class T>
__device__ __forceinline__ void encode_group(const T* __restrict__ x, int64_t step, int left,
                                             uint8_t* __restrict__ codes, uint8_t* __restrict__ scale) {
    float v[4][8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i / 8][i % 8] = i < left ? to_f32(x[i * step]) : 0.0f;
        amax = umax(amax, abs_bits(v[i / 8][i % 8]));
    }
    const uint32_t byte = mx_byte(amax);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = byte == kMxNaN ? 0u : mx_codes8(v[i], mx_scale(byte));
    *reinterpret_cast<u32x4*>(codes) = w;
    *scale = (uint8_t)byte;
}

struct Outputs {
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, dim;  // of the matrix that they hold
    int64_t pitch, spitch;
};

// ROWS: element (r, c) of the output is x[r * ldx + c], else x[c * ldx + r].
template <class T, bool ROWS>
__global__ void __launch_bounds__(256)
k_enc_mxfp4(const T* __restrict__ x, int64_t ldx, Outputs o, int64_t total) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t groups = o.spitch;  // with those that only pad the scales
        const int64_t r = ROWS ? i / groups : i % o.rows, q = ROWS ? i % groups : i / o.rows;
        const int64_t c = q * kMxGroup;
        if (c < o.dim)
            encode_group(ROWS ? x + r * ldx + c : x + c * ldx + r, ROWS ? 1 : ldx,
                         (int)(o.dim - c < kMxGroup ? o.dim - c : kMxGroup), o.codes + r * o.pitch + q * 16,
                         o.scales + r * o.spitch + q);
        else
            o.scales[r * o.spitch + q] = 0;
    }
}

template <class T>
__global__ void __launch_bounds__(256)
k_dec_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int64_t dim,
            int64_t pitch, int64_t spitch, T* __restrict__ out, int64_t ldo, int64_t total) {
    const int64_t words = pitch / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / words, q = i % words, c = q * 8;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + r * pitch + q * 4);
        const uint32_t byte = scales[r * spitch + c / kMxGroup];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t code = (w >> (4 * j)) & 15u, e = (code >> 1) & 3u;
            // the values of the codes: 1 + half the low bit, times 2^(e - 1), and 0 and 0.5 below
            const float mag = e ? __uint_as_float(((e + 126u) << 23) | ((code & 1u) << 22)) : (code & 1u) * 0.5f;
            const float scale = byte == kMxNaN ? __uint_as_float(0x7FC00000u) : mx_scale(byte);
            v[j] = (code & 8u ? -mag : mag) * scale;
        }
        store8(out + r * ldo + c, dim - c, v);
    }
}

unsigned grid_of(int64_t total) {
    const int64_t g = (total + 255) / 256;
    return (unsigned)(g < kMaxBlocks ? g : kMaxBlocks);
}

Outputs outputs(void* codes, void* scales, int64_t rows, int64_t dim) {
    return Outputs{static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, dim, (dim + 31) / 32 * 16,
                   (dim + 127) / 128 * 4};
}

template <class T>
hipError_t encode(const T* x, int64_t rows, int64_t dim, int64_t ldx, void* codes, void* scales, void* codes_t,
                  void* scales_t, hipStream_t stream) {
    if (codes) {
        const Outputs o = outputs(codes, scales, rows, dim);
        const int64_t total = rows * o.spitch;
        hipLaunchKernelGGL((k_enc_mxfp4<T, true>), dim3(grid_of(total)), dim3(256), 0, stream, x, ldx, o, total);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (codes_t) {
        const Outputs o = outputs(codes_t, scales_t, dim, rows);
        const int64_t total = dim * o.spitch;
        hipLaunchKernelGGL((k_enc_mxfp4<T, false>), dim3(grid_of(total)), dim3(256), 0, stream, x, ldx, o, total);
        return hipGetLastError();
    }
    return hipSuccess;
}

template <class T>
hipError_t decode(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t dim, T* out, int64_t ldo,
                  hipStream_t stream) {
    const int64_t pitch = (dim + 31) / 32 * 16, spitch = (dim + 127) / 128 * 4, total = rows * (pitch / 4);
    hipLaunchKernelGGL(k_dec_mxfp4<T>, dim3(grid_of(total)), dim3(256), 0, stream, codes, scales, rows, dim, pitch,
                       spitch, out, ldo, total);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_encode_mxfp4(const void* x, bool bf16, int64_t rows, int64_t dim, int64_t ldx, void* codes,
                               void* scales, void* codes_t, void* scales_t, hipStream_t stream) {
    return bf16 ? encode(static_cast<const BF16*>(x), rows, dim, ldx, codes, scales, codes_t, scales_t, stream)
                : encode(static_cast<const float*>(x), rows, dim, ldx, codes, scales, codes_t, scales_t, stream);
}

hipError_t launch_decode_mxfp4(const void* codes, const void* scales, int64_t rows, int64_t dim, void* out, bool bf16,
                               int64_t ldo, hipStream_t stream) {
    const uint8_t* c = static_cast<const uint8_t*>(codes);
    const uint8_t* s = static_cast<const uint8_t*>(scales);
    return bf16 ? decode(c, s, rows, dim, static_cast<BF16*>(out), ldo, stream)
                : decode(c, s, rows, dim, static_cast<float*>(out), ldo, stream);
}

}  // namespace qc
