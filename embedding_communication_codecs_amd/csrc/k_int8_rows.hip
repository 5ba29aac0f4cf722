// k_int8_rows.hip -- symmetric INT8 codes with one fp32 scale per row: the
// form in which activations (a row per token) and weights (a row per output
// channel) enter the INT8 matrix product.
//
// Per row: scale = fl(max|x| / 127); code = the integer nearest to the real
// quotient x / scale, ties to even.  A row with an infinity or a NaN gets
// scale NaN and codes 0; a zero scale gives codes 0.
//
// Bound by HBM (2 bytes read per byte written for bf16, 4 for fp32).  A row is
// held in registers between the two uses of its values, by one wave where it
// is short and by a block of 4 waves otherwise, so x is read once.  16384 x
// 8192 bf16: 67 us, 6.0 TB/s, fp32 115 us, 5.8; 4096 x 4096 bf16 11.5 us; one row of
// 4096 2.3 us, the latency of one load, one reduction over the block and one
// store.  Rows longer than 16,384 are read twice, from HBM both times: 4096 x
// 28672 bf16 97 us, fp32 196, which is 6.1 and 5.4 TB/s with both reads counted.
#include "qc_matrix.hpp"
#include "qc_launch.hpp"

namespace qc {
namespace {

// Sum (see kWhole) whose low byte is the code of v, for r = fl(1/s) of the
// row's scale s.  v * r is within 127 * 2^-23 (1.6e-5) of the real quotient,
// so unless it lies closer than 2e-5 to the middle between two whole
// numbers its nearest one is the right one; `far` gathers the distance from
// it, and the caller decides the exceptions in 64 bits.
__device__ __forceinline__ float code_fast(float v, float r, float& far) {
    const float sum = __builtin_fmaf(v, r, kWhole);
    far = fmaxf(far, fabsf(__builtin_fmaf(v, r, kWhole - sum)));
    return sum;
}

// In 64 bits the quotient of two fp32 numbers is a half-integer only if the
// real one is: a quotient that differs from (c + 1/2) does so by at least
// 2^-32 of it.
__device__ __forceinline__ float code_exact(float v, float s) {
    const double q = __builtin_rint((double)v / (double)s);
    return (float)fmin(fmax(q, -127.0), 127.0) + kWhole;
}

__device__ __forceinline__ uint64_t encode8(const float (&v)[8], float s, float r, bool fast) {
    float q[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = code_fast(v[i], r, far);
    const bool near = !fast || far >= 0.49998f;
    if (__any(near)) {
        if (near) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = s > 0.0f ? code_exact(v[i], s) : kWhole;
        }
    }
    return (uint64_t)low_bytes(q[0], q[1], q[2], q[3]) | ((uint64_t)low_bytes(q[4], q[5], q[6], q[7]) << 32);
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(v[i]));
    return m;
}

// Scale and reciprocal of a row from the bits of its largest magnitude.
// `fast`: the reciprocal and every product with it are normal numbers.
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float& r, bool& fast) {
    if (amax_bits >= kInfBits) {
        r = 0.0f;
        fast = false;
        return __uint_as_float(0x7FC00000u);
    }
    const float s = __uint_as_float(amax_bits) / 127.0f;
    fast = s >= 0x1p-100f;
    r = fast ? 1.0f / s : 0.0f;
    return s;
}

// A row of at most WPR * 64 * 8 * CH values, held by WPR waves: chunk c of
// thread t covers the 8 values from 8 * (c * 64 * WPR + t).
template <class T, int WPR, int CH>
__global__ void __launch_bounds__(256)
k_enc_int8_row(const T* __restrict__ x, int64_t rows, int64_t dim, int64_t ldx, uint8_t* __restrict__ codes,
               int64_t ldq, float* __restrict__ scale) {
    constexpr int TPR = WPR * WAVE, RPB = 4 / WPR;
    __shared__ uint32_t part[4];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t padded = (dim + 15) & ~int64_t(15);
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < rows; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = row0 + sub;
        const bool live = row < rows;
        const T* xr = x + row * ldx;
        float v[CH][8];
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int64_t at = 8 * (int64_t)(c * TPR + t);
            load8(xr + at, live ? dim - at : 0, v[c]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) amax = umax(amax, amax8(v[c]));
        amax = group_max_u32<WAVE>(amax);
        if constexpr (WPR > 1) {
            if (lane_id() == 0) part[wave_id()] = amax;
            __syncthreads();
            amax = umax(umax(part[0], part[1]), umax(part[2], part[3]));
            __syncthreads();  // part may be rewritten for the next row
        }
        float r;
        bool fast;
        const float s = row_scale(amax, r, fast);
        if (live) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int64_t at = 8 * (int64_t)(c * TPR + t);
                if (at < padded)
                    *reinterpret_cast<uint64_t*>(codes + row * ldq + at) = encode8(v[c], s, r, fast);
            }
            if (t == 0) scale[row] = s;
        }
    }
}

// Any longer row: one block, two passes over it.
template <class T>
__global__ void __launch_bounds__(256)
k_enc_int8_long(const T* __restrict__ x, int64_t rows, int64_t dim, int64_t ldx, uint8_t* __restrict__ codes,
                int64_t ldq, float* __restrict__ scale) {
    __shared__ uint32_t part[4];
    const int64_t padded = (dim + 15) & ~int64_t(15);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + row * ldx;
        uint32_t amax = 0;
        for (int64_t at = 8 * (int64_t)threadIdx.x; at < dim; at += 2048) {
            float v[8];
            load8(xr + at, dim - at, v);
            amax = umax(amax, amax8(v));
        }
        amax = group_max_u32<WAVE>(amax);
        if (lane_id() == 0) part[wave_id()] = amax;
        __syncthreads();
        amax = umax(umax(part[0], part[1]), umax(part[2], part[3]));
        __syncthreads();
        float r;
        bool fast;
        const float s = row_scale(amax, r, fast);
        for (int64_t at = 8 * (int64_t)threadIdx.x; at < padded; at += 2048) {
            float v[8];
            load8(xr + at, dim - at, v);
            *reinterpret_cast<uint64_t*>(codes + row * ldq + at) = encode8(v, s, r, fast);
        }
        if (threadIdx.x == 0) scale[row] = s;
    }
}

template <class T, int WPR, int CH>
hipError_t launch_row(const T* x, int64_t rows, int64_t dim, int64_t ldx, uint8_t* codes, int64_t ldq, float* scale,
                      hipStream_t stream) {
    constexpr int RPB = 4 / WPR;
    const int64_t blocks = (rows + RPB - 1) / RPB;
    hipLaunchKernelGGL((k_enc_int8_row<T, WPR, CH>), dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)),
                       dim3(256), 0, stream, x, rows, dim, ldx, codes, ldq, scale);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const T* x, int64_t rows, int64_t dim, int64_t ldx, uint8_t* codes, int64_t ldq, float* scale,
                  hipStream_t stream) {
    // By a row's length alone: a wave holds up to 1,024 values, 16 a lane; a
    // block's four waves up to 16,384, 64 a lane.
    if (dim <= 512) return launch_row<T, 1, 1>(x, rows, dim, ldx, codes, ldq, scale, stream);
    if (dim <= 1024) return launch_row<T, 1, 2>(x, rows, dim, ldx, codes, ldq, scale, stream);
    if (dim <= 2048) return launch_row<T, 4, 1>(x, rows, dim, ldx, codes, ldq, scale, stream);
    if (dim <= 4096) return launch_row<T, 4, 2>(x, rows, dim, ldx, codes, ldq, scale, stream);
    if (dim <= 8192) return launch_row<T, 4, 4>(x, rows, dim, ldx, codes, ldq, scale, stream);
    if (dim <= 16384) return launch_row<T, 4, 8>(x, rows, dim, ldx, codes, ldq, scale, stream);
    hipLaunchKernelGGL(k_enc_int8_long<T>, dim3((unsigned)(rows < kMaxBlocks ? rows : kMaxBlocks)), dim3(256), 0,
                       stream, x, rows, dim, ldx, codes, ldq, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_encode_int8_rowwise(const void* x, bool bf16, int64_t rows, int64_t dim, int64_t ldx, void* codes,
                                      int64_t ldq, float* scale, hipStream_t stream) {
    uint8_t* q = static_cast<uint8_t*>(codes);
    if (bf16) return launch(static_cast<const BF16*>(x), rows, dim, ldx, q, ldq, scale, stream);
    return launch(static_cast<const float*>(x), rows, dim, ldx, q, ldq, scale, stream);
}

}  // namespace qc
