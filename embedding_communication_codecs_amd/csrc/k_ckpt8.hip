// k_ckpt8.hip -- matrices held in 8 bits between the forward and the
// backward pass ("checkpoints"), and the gated activation that keeps two.
//
// A checkpoint holds each group of 32 consecutive values of a row as INT8
// codes q with one power-of-two step 2^E (qc_matrix.hpp, ckpt_byte): 1 +
// 1/32 bytes a value.  q * 2^E is exact in bf16 as well as in fp32, so what
// a backward pass reads is a bf16 matrix that was never rounded again.
//
// All of this is bound by HBM.  16 lanes hold 128 consecutive values of a
// row, 8 each (one 16-byte load of bf16): a group is four lanes, its largest
// magnitude two DPP steps away, and the four exponent bytes of the 128 values
// leave as one word.  8192 x 8192 bf16: save and restore 34.5 us each, 5.9
// TB/s; the gated activation 88 us forward and 85 backward, 6.2 and 6.4 TB/s.
#include "qc_matrix.hpp"
#include "qc_launch.hpp"

namespace qc {
namespace {

struct Kept {  // a checkpoint's buffers
    uint8_t* codes;
    uint8_t* exps;
};
struct KeptIn {
    const uint8_t* codes;
    const uint8_t* exps;
};

// Where a thread works: 16 lanes are a unit of 128 columns, a block of 256
// threads holds 16 units, 2^lx of them side by side and the others in rows
// below, so narrow matrices fill blocks too.  Grid: x the tiles of a row, y
// the tiles of rows.  Saving and restoring take two of the latter at a time,
// with the loads of both before the first use (8192 x 8192 bf16: save 34.3
// us against 38.4 with one and 34.4 with four, restore 34.6 against 35.3 and
// 35.7); the gated activation, which holds more, takes one (backward 87 us
// against 92 with two).
constexpr int kUnroll = 2;
struct Place {
    int64_t row, col;
    bool live;  // the unit has values (its lanes may still be past dim)
};

struct Sizes {
    int64_t rows, dim, pitch, epitch, row_tiles;
    int lx;
};

__device__ __forceinline__ Place place_of(int64_t rt, const Sizes& z) {
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t row = (rt << (4 - z.lx)) + (unit >> z.lx);
    const int64_t u = ((int64_t)blockIdx.x << z.lx) + (unit & ((1 << z.lx) - 1));
    return Place{row, u * 128 + 8 * l, row < z.rows && u * 128 < z.dim};
}

// The exponent bytes of a unit's four groups, gathered into lane 0 of its 16
// (row_shl:n reads lane i + n).
__device__ __forceinline__ uint32_t gather_bytes(uint32_t b) {
    const uint32_t b1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x104, 0xF, 0xF, true);
    const uint32_t b2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x108, 0xF, 0xF, true);
    const uint32_t b3 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x10C, 0xF, 0xF, true);
    return b | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

// Every lane of the wave calls this (lanes without values hold zeros).
__device__ __forceinline__ void keep8(const float (&v)[8], const Place& p, const Sizes& z, const Kept& k) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = umax(amax, abs_bits(v[i]));
    amax = quad_max(amax);
    const bool group = p.live && (p.col & ~int64_t(31)) < z.dim;  // else: padding, byte 0
    const uint32_t byte = group ? ckpt_byte(amax) : 0u;
    const uint32_t word = gather_bytes(byte);
    if (p.live && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(k.exps + p.row * z.epitch + p.col / 32) = word;
    if (group) {
        const u32x2 w = ckpt_codes(v, byte);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(k.codes + p.row * z.pitch + p.col));
    }
}

struct Raw8 {  // 8 codes and their step's byte
    u32x2 codes;
    uint32_t byte;
};
__device__ __forceinline__ Raw8 held_raw8(const KeptIn& k, const Place& p, const Sizes& z) {
    if (!(p.live && p.col < z.dim)) return Raw8{u32x2{0, 0}, 0};
    return Raw8{ld_stream_u2(k.codes + p.row * z.pitch + p.col), k.exps[p.row * z.epitch + p.col / 32]};
}
__device__ __forceinline__ int64_t left_of(const Place& p, const Sizes& z) { return p.live ? z.dim - p.col : 0; }

template <class T>
__global__ void __launch_bounds__(256)
k_enc_ckpt8(const T* __restrict__ x, int64_t ldx, Sizes z, Kept k) {
    constexpr int U = kUnroll;
    for (int64_t rt = (int64_t)blockIdx.y * U; rt < z.row_tiles; rt += (int64_t)gridDim.y * U) {
        float v[U][8];
        Place p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = place_of(rt + u, z);
            load8(x + p[u].row * ldx + p[u].col, left_of(p[u], z), v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) keep8(v[u], p[u], z, k);
    }
}

template <class T>
__global__ void __launch_bounds__(256)
k_dec_ckpt8(KeptIn k, Sizes z, T* __restrict__ out, int64_t ldo) {
    constexpr int U = kUnroll;
    for (int64_t rt = (int64_t)blockIdx.y * U; rt < z.row_tiles; rt += (int64_t)gridDim.y * U) {
        Raw8 r[U];
        Place p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = place_of(rt + u, z);
            r[u] = held_raw8(k, p[u], z);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            ckpt_values(r[u].codes, r[u].byte, v);
            store8(out + p[u].row * ldo + p[u].col, left_of(p[u], z), v);
        }
    }
}

// s = 1 / (1 + exp(-x)) and c = 1 - s.  With a = exp(-|x|), in (0, 1], r =
// 1 / (1 + a): r and a * r are the two of them, the larger first, neither
// from a difference.  -|x| log2 e = n + f with n the nearest integer and f
// from multiply-adds with log2 e's two parts, so that a = 2^f 2^n has a relative
// error that does not grow with |x|.  The scaling by 2^n is apart, as the
// hardware's 2^y is 0 where its result is below 2^-126: gates from -87 to -103
// have a sigmoid that another factor can make a normal number.  r takes one
// Newton step from the hardware's reciprocal.  About 22 issue slots against
// 45 with expf and divisions, which the forward pass was bound by (8192 x
// 8192: 106 us).
__device__ __forceinline__ void sigmoid(float x, float& s, float& c) {
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0c0p-26f;
    const float m = fminf(fabsf(x), 130.0f);  // n stays above -188
    const float sum = __builtin_fmaf(m, -kLog2e, kWhole), n = sum - kWhole;
    const float f = __builtin_fmaf(m, -kLog2eLow, __builtin_fmaf(m, -kLog2e, -n));
    // 2^(n + 64), whose exponent field comes from the sum's low bits, then 2^-64
    const float up = __uint_as_float((__float_as_uint(sum) + (127u + 64u)) << 23);
    const float a = __builtin_amdgcn_exp2f(f) * up * 0x1p-64f;
    const float q = 1.0f + a, r0 = __builtin_amdgcn_rcpf(q);
    const float r = __builtin_fmaf(__builtin_fmaf(-q, r0, 1.0f), r0, r0);
    const float ar = a * r;
    s = x < 0.0f ? ar : r;
    c = x < 0.0f ? r : ar;
}

// h = silu(g) * u, and the checkpoints of g and u.
template <class T>
__global__ void __launch_bounds__(256)
k_swiglu_ckpt8(const T* __restrict__ gate, const T* __restrict__ up, int64_t ldx, Sizes z, T* __restrict__ h,
               int64_t ldh, Kept kg, Kept ku) {
    for (int64_t rt = blockIdx.y; rt < z.row_tiles; rt += gridDim.y) {
        const Place p = place_of(rt, z);
        float g[8], u[8];
        load8(gate + p.row * ldx + p.col, left_of(p, z), g);
        load8(up + p.row * ldx + p.col, left_of(p, z), u);
        keep8(g, p, z, kg);
        keep8(u, p, z, ku);
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s, c;
            sigmoid(g[e], s, c);
            o[e] = g[e] * s * u[e];
        }
        store8(h + p.row * ldh + p.col, left_of(p, z), o);
    }
}

// With G, U as held and s = 1 / (1 + exp(-G)):
//   dU = dh * G * s,  dG = dh * U * s * (1 + G * (1 - s)).
template <class T>
__global__ void __launch_bounds__(256)
k_swiglu_ckpt8_bwd(const T* __restrict__ dh, int64_t lddh, KeptIn kg, KeptIn ku, Sizes z, T* __restrict__ dgate,
                   T* __restrict__ dup, int64_t ldg) {
    for (int64_t rt = blockIdx.y; rt < z.row_tiles; rt += gridDim.y) {
        const Place p = place_of(rt, z);
        float d[8], g[8], u[8];
        load8(dh + p.row * lddh + p.col, left_of(p, z), d);
        const Raw8 rg = held_raw8(kg, p, z), ru = held_raw8(ku, p, z);
        ckpt_values(rg.codes, rg.byte, g);
        ckpt_values(ru.codes, ru.byte, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s, c;
            sigmoid(g[e], s, c);
            // silu's derivative first: it is never above 1.1, where dh * U may
            // overflow, and a subnormal s is rounded no further before it is scaled
            const float a = d[e] * (s * (1.0f + g[e] * c)) * u[e];
            u[e] = d[e] * s * g[e];
            g[e] = a;
        }
        store8(dgate + p.row * ldg + p.col, left_of(p, z), g);
        store8(dup + p.row * ldg + p.col, left_of(p, z), u);
    }
}

struct Launch {
    Sizes z;
    dim3 grid;
};

// `unroll`: tiles of rows that a thread takes at a time
Launch launch_of(int64_t rows, int64_t dim, int unroll) {
    Launch n;
    const int64_t units = (dim + 127) / 128;
    n.z.rows = rows;
    n.z.dim = dim;
    n.z.lx = units >= 16 ? 4 : log2_exact(units);
    n.z.pitch = (dim + 31) / 32 * 32;
    n.z.epitch = units * 4;
    n.z.row_tiles = (rows + (16 >> n.z.lx) - 1) >> (4 - n.z.lx);
    const int64_t y = (n.z.row_tiles + unroll - 1) / unroll;
    n.grid = dim3((unsigned)((units + (1 << n.z.lx) - 1) >> n.z.lx), (unsigned)(y < 65535 ? y : 65535));
    return n;
}

template <class T>
hipError_t enc(const void* x, int64_t ldx, int64_t rows, int64_t dim, Kept k, hipStream_t stream) {
    const Launch n = launch_of(rows, dim, kUnroll);
    hipLaunchKernelGGL((k_enc_ckpt8<T>), n.grid, dim3(256), 0, stream, static_cast<const T*>(x), ldx, n.z, k);
    return hipGetLastError();
}

template <class T>
hipError_t dec(KeptIn k, int64_t rows, int64_t dim, void* out, int64_t ldo, hipStream_t stream) {
    const Launch n = launch_of(rows, dim, kUnroll);
    hipLaunchKernelGGL((k_dec_ckpt8<T>), n.grid, dim3(256), 0, stream, k, n.z, static_cast<T*>(out), ldo);
    return hipGetLastError();
}

template <class T>
hipError_t swiglu(const void* gate, const void* up, int64_t ldx, int64_t rows, int64_t dim, void* h, int64_t ldh,
                  Kept kg, Kept ku, hipStream_t stream) {
    const Launch n = launch_of(rows, dim, 1);
    hipLaunchKernelGGL((k_swiglu_ckpt8<T>), n.grid, dim3(256), 0, stream, static_cast<const T*>(gate),
                       static_cast<const T*>(up), ldx, n.z, static_cast<T*>(h), ldh, kg, ku);
    return hipGetLastError();
}

template <class T>
hipError_t swiglu_bwd(const void* dh, int64_t lddh, KeptIn kg, KeptIn ku, int64_t rows, int64_t dim, void* dgate,
                      void* dup, int64_t ldg, hipStream_t stream) {
    const Launch n = launch_of(rows, dim, 1);
    hipLaunchKernelGGL((k_swiglu_ckpt8_bwd<T>), n.grid, dim3(256), 0, stream, static_cast<const T*>(dh), lddh, kg,
                       ku, n.z, static_cast<T*>(dgate), static_cast<T*>(dup), ldg);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_encode_ckpt8(const void* x, bool bf16, int64_t ldx, int64_t rows, int64_t dim, void* codes,
                               void* exps, hipStream_t stream) {
    const Kept k{static_cast<uint8_t*>(codes), static_cast<uint8_t*>(exps)};
    return bf16 ? enc<BF16>(x, ldx, rows, dim, k, stream) : enc<float>(x, ldx, rows, dim, k, stream);
}

hipError_t launch_decode_ckpt8(const void* codes, const void* exps, int64_t rows, int64_t dim, void* out, bool bf16,
                               int64_t ldo, hipStream_t stream) {
    const KeptIn k{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(exps)};
    return bf16 ? dec<BF16>(k, rows, dim, out, ldo, stream) : dec<float>(k, rows, dim, out, ldo, stream);
}

hipError_t launch_swiglu_ckpt8(const void* gate, const void* up, bool bf16, int64_t ldx, int64_t rows, int64_t dim,
                               void* h, int64_t ldh, void* gate_codes, void* gate_exps, void* up_codes,
                               void* up_exps, hipStream_t stream) {
    const Kept kg{static_cast<uint8_t*>(gate_codes), static_cast<uint8_t*>(gate_exps)};
    const Kept ku{static_cast<uint8_t*>(up_codes), static_cast<uint8_t*>(up_exps)};
    return bf16 ? swiglu<BF16>(gate, up, ldx, rows, dim, h, ldh, kg, ku, stream)
                : swiglu<float>(gate, up, ldx, rows, dim, h, ldh, kg, ku, stream);
}

hipError_t launch_swiglu_ckpt8_backward(const void* dh, bool bf16, int64_t lddh, const void* gate_codes,
                                        const void* gate_exps, const void* up_codes, const void* up_exps,
                                        int64_t rows, int64_t dim, void* dgate, void* dup, int64_t ldg,
                                        hipStream_t stream) {
    const KeptIn kg{static_cast<const uint8_t*>(gate_codes), static_cast<const uint8_t*>(gate_exps)};
    const KeptIn ku{static_cast<const uint8_t*>(up_codes), static_cast<const uint8_t*>(up_exps)};
    return bf16 ? swiglu_bwd<BF16>(dh, lddh, kg, ku, rows, dim, dgate, dup, ldg, stream)
                : swiglu_bwd<float>(dh, lddh, kg, ku, rows, dim, dgate, dup, ldg, stream);
}

}  // namespace qc
