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
// leave as one word.
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
// below, so narrow matrices fill blocks too.
struct Place {
    int64_t row, col;
    bool live;  // the unit has values (its lanes may still be past dim)
};

__device__ __forceinline__ Place place_of(int64_t tile, int64_t rows, int64_t dim, int lx, int64_t col_tiles) {
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t rt = tile / col_tiles, ct = tile - rt * col_tiles;
    const int64_t row = (rt << (4 - lx)) + (unit >> lx);
    const int64_t u = (ct << lx) + (unit & ((1 << lx) - 1));
    return Place{row, u * 128 + 8 * l, row < rows && u * 128 < dim};
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
__device__ __forceinline__ void keep8(const float (&v)[8], const Place& p, int64_t dim, const Kept& k,
                                      int64_t pitch, int64_t epitch) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = umax(amax, abs_bits(v[i]));
    amax = quad_max(amax);
    const bool group = p.live && (p.col & ~int64_t(31)) < dim;  // else: padding, byte 0
    const uint32_t byte = group ? ckpt_byte(amax) : 0u;
    const uint32_t word = gather_bytes(byte);
    if (p.live && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(k.exps + p.row * epitch + p.col / 32) = word;
    if (group) {
        const float inv = __uint_as_float((254u - min(byte, 254u)) << 23);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = byte == kCkptNaN ? 0.0f : ckpt_code(v[i], inv);
        const u32x2 w = {pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(k.codes + p.row * pitch + p.col));
    }
}

__device__ __forceinline__ void held8(const KeptIn& k, const Place& p, int64_t pitch, int64_t epitch, float (&v)[8]) {
    const u32x2 w = ld_stream_u2(k.codes + p.row * pitch + p.col);
    const float step = ckpt_step(k.exps[p.row * epitch + p.col / 32]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * step;
}

template <class T>
__global__ void __launch_bounds__(256)
k_enc_ckpt8(const T* __restrict__ x, int64_t ldx, int64_t rows, int64_t dim, int lx, int64_t col_tiles, int64_t tiles,
            Kept k, int64_t pitch, int64_t epitch) {
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Place p = place_of(tile, rows, dim, lx, col_tiles);
        float v[8];
        load8(x + p.row * ldx + p.col, p.live ? dim - p.col : 0, v);
        keep8(v, p, dim, k, pitch, epitch);
    }
}

template <class T>
__global__ void __launch_bounds__(256)
k_dec_ckpt8(KeptIn k, int64_t pitch, int64_t epitch, int64_t rows, int64_t dim, int lx, int64_t col_tiles,
            int64_t tiles, T* __restrict__ out, int64_t ldo) {
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Place p = place_of(tile, rows, dim, lx, col_tiles);
        if (p.live && p.col < dim) {
            float v[8];
            held8(k, p, pitch, epitch, v);
            store8(out + p.row * ldo + p.col, dim - p.col, v);
        }
    }
}

// h = silu(g) * u, and the checkpoints of g and u.
template <class T>
__global__ void __launch_bounds__(256)
k_swiglu_ckpt8(const T* __restrict__ gate, const T* __restrict__ up, int64_t ldx, int64_t rows, int64_t dim, int lx,
               int64_t col_tiles, int64_t tiles, T* __restrict__ h, int64_t ldh, Kept kg, Kept ku, int64_t pitch,
               int64_t epitch) {
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Place p = place_of(tile, rows, dim, lx, col_tiles);
        const int64_t left = p.live ? dim - p.col : 0;
        float g[8], u[8];
        load8(gate + p.row * ldx + p.col, left, g);
        load8(up + p.row * ldx + p.col, left, u);
        keep8(g, p, dim, kg, pitch, epitch);
        keep8(u, p, dim, ku, pitch, epitch);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = g[i] / (1.0f + expf(-g[i])) * u[i];
        store8(h + p.row * ldh + p.col, left, o);
    }
}

// With G, U as held and s = 1 / (1 + exp(-G)):
//   dU = dh * G * s,  dG = dh * U * s * (1 + G * (1 - s)).
template <class T>
__global__ void __launch_bounds__(256)
k_swiglu_ckpt8_bwd(const T* __restrict__ dh, int64_t lddh, KeptIn kg, KeptIn ku, int64_t pitch, int64_t epitch,
                   int64_t rows, int64_t dim, int lx, int64_t col_tiles, int64_t tiles, T* __restrict__ dgate,
                   T* __restrict__ dup, int64_t ldg) {
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Place p = place_of(tile, rows, dim, lx, col_tiles);
        if (p.live && p.col < dim) {
            const int64_t left = dim - p.col;
            float d[8], g[8], u[8];
            load8(dh + p.row * lddh + p.col, left, d);
            held8(kg, p, pitch, epitch, g);
            held8(ku, p, pitch, epitch, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = 1.0f / (1.0f + expf(-g[i]));
                const float a = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
                u[i] = d[i] * g[i] * s;
                g[i] = a;
            }
            store8(dgate + p.row * ldg + p.col, left, g);
            store8(dup + p.row * ldg + p.col, left, u);
        }
    }
}

struct Tiling {
    int lx;
    int64_t col_tiles, tiles, pitch, epitch;
    dim3 grid() const { return dim3((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks)); }
};

Tiling tiling(int64_t rows, int64_t dim) {
    Tiling t;
    const int64_t units = (dim + 127) / 128;
    t.lx = units >= 16 ? 4 : log2_exact(units);
    t.col_tiles = (units + (1 << t.lx) - 1) >> t.lx;
    const int64_t rpb = 16 >> t.lx;
    t.tiles = (rows + rpb - 1) / rpb * t.col_tiles;
    t.pitch = (dim + 31) / 32 * 32;
    t.epitch = units * 4;
    return t;
}

template <class T>
hipError_t enc(const void* x, int64_t ldx, int64_t rows, int64_t dim, Kept k, hipStream_t stream) {
    const Tiling t = tiling(rows, dim);
    hipLaunchKernelGGL(k_enc_ckpt8<T>, t.grid(), dim3(256), 0, stream, static_cast<const T*>(x), ldx, rows, dim, t.lx,
                       t.col_tiles, t.tiles, k, t.pitch, t.epitch);
    return hipGetLastError();
}

template <class T>
hipError_t dec(KeptIn k, int64_t rows, int64_t dim, void* out, int64_t ldo, hipStream_t stream) {
    const Tiling t = tiling(rows, dim);
    hipLaunchKernelGGL(k_dec_ckpt8<T>, t.grid(), dim3(256), 0, stream, k, t.pitch, t.epitch, rows, dim, t.lx,
                       t.col_tiles, t.tiles, static_cast<T*>(out), ldo);
    return hipGetLastError();
}

template <class T>
hipError_t swiglu(const void* gate, const void* up, int64_t ldx, int64_t rows, int64_t dim, void* h, int64_t ldh,
                  Kept kg, Kept ku, hipStream_t stream) {
    const Tiling t = tiling(rows, dim);
    hipLaunchKernelGGL(k_swiglu_ckpt8<T>, t.grid(), dim3(256), 0, stream, static_cast<const T*>(gate),
                       static_cast<const T*>(up), ldx, rows, dim, t.lx, t.col_tiles, t.tiles, static_cast<T*>(h), ldh,
                       kg, ku, t.pitch, t.epitch);
    return hipGetLastError();
}

template <class T>
hipError_t swiglu_bwd(const void* dh, int64_t lddh, KeptIn kg, KeptIn ku, int64_t rows, int64_t dim, void* dgate,
                      void* dup, int64_t ldg, hipStream_t stream) {
    const Tiling t = tiling(rows, dim);
    hipLaunchKernelGGL(k_swiglu_ckpt8_bwd<T>, t.grid(), dim3(256), 0, stream, static_cast<const T*>(dh), lddh, kg, ku,
                       t.pitch, t.epitch, rows, dim, t.lx, t.col_tiles, t.tiles, static_cast<T*>(dgate),
                       static_cast<T*>(dup), ldg);
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
