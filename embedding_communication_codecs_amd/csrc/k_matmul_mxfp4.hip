// k_matmul_mxfp4.hip -- C[m][n] (+)= sum over k of A[m][k] B[n][k], both in
// MXFP4 with k contiguous: tokens (A) and weights (B).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 rows x 64 values of each side, a
// lane one group of 32 of a row with its scale byte, and accumulates in fp32.
// The weights are its first operand and the tokens its second, so a lane ends
// up with four times four neighbouring output channels of one token.
#include "qc_launch.hpp"
#include "qc_mx.hpp"

namespace qc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Side {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;
};
struct Args {
    Side a, b;  // tokens, weights
    int64_t pitch, spitch, k;
    int64_t ldc;
};

__device__ __forceinline__ i32x8 operand(u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

template <class T, bool ADD>
__global__ void __launch_bounds__(64)
k_mm_mxfp4(Args g, T* __restrict__ c) {
    const int64_t tn = (g.b.rows + 31) / 32;
    const int64_t n0 = (int64_t)(blockIdx.x % tn) * 32, m0 = (int64_t)(blockIdx.x / tn) * 32;
    const int l = lane_id(), half = l >> 5;
    const int64_t rb = min(n0 + (l & 31), g.b.rows - 1), ra = min(m0 + (l & 31), g.a.rows - 1);
    f32x16 acc = {};
    for (int64_t q = 0; q * 64 < g.k; ++q) {
        const int64_t group = 2 * q + half;
        u32x4 fa = {0, 0, 0, 0}, fb = {0, 0, 0, 0};
        int sa = 127, sb = 127;
        if (group * 16 < g.pitch) {
            fa = ld_u4(g.a.codes + ra * g.pitch + group * 16);
            fb = ld_u4(g.b.codes + rb * g.pitch + group * 16);
            sa = g.a.scales[ra * g.spitch + group];
            sb = g.b.scales[rb * g.spitch + group];
        }
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb), operand(fa), acc, 4, 4, 0, sb, 0, sa);
    }
    const int64_t row = m0 + (l & 31);
    if (row >= g.a.rows) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int64_t col = n0 + 8 * (e / 4) + 4 * half + e % 4;
        if (col < g.b.rows) {
            T* p = c + row * g.ldc + col;
            if constexpr (ADD) *p = *p + acc[e];
            else put(p, acc[e]);
        }
    }
}

}  // namespace

int64_t matmul_mxfp4_workspace(int64_t m, int64_t n, int64_t k) {
    (void)m, (void)n, (void)k;
    return 0;
}

hipError_t launch_matmul_mxfp4(const void* a, const void* a_scales, const void* b, const void* b_scales, int64_t m,
                               int64_t n, int64_t k, void* c, bool bf16, int64_t ldc, bool accumulate,
                               void* workspace, hipStream_t stream) {
    (void)workspace;
    const Args g{{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales), m},
                 {static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales), n},
                 (k + 31) / 32 * 16, (k + 127) / 128 * 4, k, ldc};
    const dim3 grid((unsigned)(((n + 31) / 32) * ((m + 31) / 32)));
    if (bf16)
        hipLaunchKernelGGL((k_mm_mxfp4<BF16, false>), grid, dim3(64), 0, stream, g, static_cast<BF16*>(c));
    else if (accumulate)
        hipLaunchKernelGGL((k_mm_mxfp4<float, true>), grid, dim3(64), 0, stream, g, static_cast<float*>(c));
    else
        hipLaunchKernelGGL((k_mm_mxfp4<float, false>), grid, dim3(64), 0, stream, g, static_cast<float*>(c));
    return hipGetLastError();
}

// Codes of x, then their scales, each from a multiple of 256 bytes on; then the product's own.
namespace {
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }
}  // namespace

int64_t linear_mxfp4_workspace(int64_t m, int64_t n, int64_t k, bool x_bf16) {
    (void)x_bf16;
    return up256(m * ((k + 31) / 32 * 16)) + up256(m * ((k + 127) / 128 * 4)) + matmul_mxfp4_workspace(m, n, k);
}

hipError_t launch_linear_mxfp4(const void* x, bool x_bf16, int64_t ldx, const void* b, const void* b_scales, int64_t m,
                               int64_t n, int64_t k, void* c, bool bf16, int64_t ldc, void* workspace,
                               hipStream_t stream) {
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + up256(m * ((k + 31) / 32 * 16));
    uint8_t* rest = scales + up256(m * ((k + 127) / 128 * 4));
    const hipError_t e = launch_encode_mxfp4(x, x_bf16, m, k, ldx, codes, scales, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    return launch_matmul_mxfp4(codes, scales, b, b_scales, m, n, k, c, bf16, ldc, false, rest, stream);
}

}  // namespace qc
