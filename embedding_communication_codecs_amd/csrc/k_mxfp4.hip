// k_mxfp4.hip -- matrices to MXFP4 and back: codes and scale bytes of a matrix
// and of its transpose (qc_mx.hpp has the format's rules).
//
// All of this is bound by HBM: 2 or 4 bytes a value on one side, 1/2 + 1/32 for
// each of the encodings on the other.  8192 x 8192, where a copy moves 5.2 TB/s:
// rows from bf16 30 us, 5.7 TB/s, from fp32 57 us, 5.3; decoded to bf16 28 us,
// 6.1 (part of the codes lies in the last cache), to fp32 52 us, 5.8.
#include "qc_launch.hpp"
#include "qc_lds.hpp"
#include "qc_mx.hpp"

#include <type_traits>

namespace qc {
namespace {

struct Coded {  // an encoding's buffers
    uint8_t* codes;
    uint8_t* scales;
    int64_t pitch, spitch;
};

// ------------------------------------------------------------------- rows
// 16 lanes are a unit of 128 columns, 8 values each: a group is four lanes, the
// four scale bytes of a unit leave as one word.  A block of 256 threads holds
// 16 units, 2^lx of them side by side and the others in rows below, so narrow
// matrices fill blocks too; each thread takes two such tiles of rows at a time,
// with the loads of both before the first use.
constexpr int kUnroll = 2;
struct Sizes {
    int64_t rows, dim, row_tiles;
    int lx;
};
struct Place {
    int64_t row, col;
    bool live;  // the unit has values (its lanes may still be past dim)
};
__device__ __forceinline__ Place place_of(int64_t rt, const Sizes& z) {
    const int unit = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t row = (rt << (4 - z.lx)) + (unit >> z.lx);
    const int64_t u = ((int64_t)blockIdx.x << z.lx) + (unit & ((1 << z.lx) - 1));
    return Place{row, u * 128 + 8 * l, row < z.rows && u * 128 < z.dim};
}
__device__ __forceinline__ int64_t left_of(const Place& p, const Sizes& z) { return p.live ? z.dim - p.col : 0; }

// The bytes of a unit's four groups, gathered into lane 0 of its 16 (row_shl:n
// reads lane i + n).
__device__ __forceinline__ uint32_t gather_bytes(uint32_t b) {
    const uint32_t b1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x104, 0xF, 0xF, true);
    const uint32_t b2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x108, 0xF, 0xF, true);
    const uint32_t b3 = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x10C, 0xF, 0xF, true);
    return b | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

// Eight values of a unit's lane; every lane of the wave calls this.
template <bool ALL, class T>
__device__ __forceinline__ void keep_row8(const Raw8<T>& v, int64_t row, int64_t col, bool live, int64_t dim,
                                          const Coded& k) {
    const uint32_t byte_here = mx_byte(quad_max(v.amax_bits()));
    live = ALL || live;
    const bool group = ALL || (live && (col & ~int64_t(31)) < dim);  // else: padding, byte 0
    const uint32_t byte = group ? byte_here : 0u;
    const uint32_t word = gather_bytes(byte);
    if (live && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(k.scales + row * k.spitch + col / 32) = word;
    if (group) {
        const uint32_t w = v.codes(mx_scale(byte));
        *reinterpret_cast<uint32_t*>(k.codes + row * k.pitch + col / 2) = byte == kMxNaN ? 0u : w;
    }
}

template <class T>
__global__ void __launch_bounds__(256)
k_enc_mxfp4(const T* __restrict__ x, int64_t ldx, Sizes z, Coded k) {
    constexpr int U = kUnroll;
    for (int64_t rt = (int64_t)blockIdx.y * U; rt < z.row_tiles; rt += (int64_t)gridDim.y * U) {
        Raw8<T> v[U];
        Place p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = place_of(rt + u, z);
            v[u].template load<true>(x + p[u].row * ldx + p[u].col, left_of(p[u], z), p[u].col > 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].settle(left_of(p[u], z), p[u].col > 0);
#pragma unroll
        for (int u = 0; u < U; ++u) keep_row8<false>(v[u], p[u].row, p[u].col, p[u].live, z.dim, k);
    }
}

// ---------------------------------------------------------------- columns
// The transpose's encoding, with or without the matrix's own: tiles of 128 x
// 128 through LDS, 512 threads each. A thread loads four pieces of 8 values
// (and encodes them by rows from its registers); then it takes 2 columns x 16
// rows, half a group of each, whose other half its neighbour has, and their
// codes leave through LDS again, 64 bytes of a row of the transpose side by
// side. Both encodings of 8192 x 8192: bf16 48 us, 4.3 TB/s, fp32 67 us, 5.1;
// the transpose's alone 37 us, 4.6, and 59 us, 5.1. (With 256 threads and whole
// groups, whose waves have twice the instructions, 1 and 4 us more, and 1027 x
// 770 6.0 and 6.6 us against 4.8 and 5.5; with 1024 as long. 1027 x 770 is 63
// tiles, so three quarters of the compute units have none. Tiles inside the
// matrix look at no bounds: 1.5 and 4.5 us. Tiles of 256 rows, whose codes
// leave 128 bytes side by side, take 44 us for this bf16 matrix, but 34.2
// against 33.6 for 8192 x 6144, 33.8 against 32.2 for 4096 x 11008, and 16.0
// against 13.6 for 4096 x 4096.)
constexpr int kTile = 128, kHalfGroup = 16;

// Byte of a row of the tile in LDS.  A wave reads 32 pairs of columns in two
// rows, 16 apart, at a time: for bf16 the 128 bytes of one lie in the other
// banks.
template <class T>
__device__ __forceinline__ int in_tile(int row, int byte) {
    const int swap = sizeof(T) == 2 ? (row / kHalfGroup & 1) << 7 : 0;
    return row * kTile * (int)sizeof(T) + (byte ^ swap);
}

template <class T>
struct Columns;  // two columns x 16 rows
template <>
struct Columns<BF16> {
    uint32_t w[kHalfGroup];
    __device__ __forceinline__ void read(const uint8_t* tile, int row0, int pair) {
#pragma unroll
        for (int r = 0; r < kHalfGroup; ++r)
            w[r] = *reinterpret_cast<const uint32_t*>(tile + in_tile<BF16>(row0, pair * 4) + r * 256);
    }
    __device__ __forceinline__ void amax_bits(uint32_t (&m)[2]) const {
        uint32_t a = 0;
#pragma unroll
        for (int r = 0; r < kHalfGroup; ++r) a = pair_max(a, w[r]);
        m[0] = a << 16;
        m[1] = a & 0xFFFF0000u;
    }
    __device__ __forceinline__ uint32_t codes8(int q, int c, float scale) const {
        const uint32_t pick = c ? 0x07060302u : 0x05040100u;  // that column's halves of two words
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_perm(w[8 * q + 2 * i + 1], w[8 * q + 2 * i], pick);
        return mx_codes8(v, scale);
    }
};
template <>
struct Columns<float> {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 w[kHalfGroup];
    __device__ __forceinline__ void read(const uint8_t* tile, int row0, int pair) {
#pragma unroll
        for (int r = 0; r < kHalfGroup; ++r)
            w[r] = *reinterpret_cast<const f32x2*>(tile + in_tile<float>(row0, pair * 8) + r * 512);
    }
    __device__ __forceinline__ void amax_bits(uint32_t (&m)[2]) const {
        m[0] = m[1] = 0;
#pragma unroll
        for (int r = 0; r < kHalfGroup; ++r) {
            m[0] = umax(m[0], abs_bits(w[r][0]));
            m[1] = umax(m[1], abs_bits(w[r][1]));
        }
    }
    __device__ __forceinline__ uint32_t codes8(int q, int c, float scale) const {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[8 * q + i][c];
        return mx_codes8(v, scale);
    }
};

__device__ __forceinline__ uint32_t pair_of_lanes_max(uint32_t v) {
    return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // quad_perm 1 0 3 2
}

__device__ __forceinline__ void put_raw8(uint8_t* tile, int row, int col, const Raw8<BF16>& v) {
    *reinterpret_cast<u32x4*>(tile + in_tile<BF16>(row, col * 2)) = v.w;
}
__device__ __forceinline__ void put_raw8(uint8_t* tile, int row, int col, const Raw8<float>& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4*>(tile + in_tile<float>(row, col * 4 + 16 * h)) =
            f32x4{v.v[4 * h], v.v[4 * h + 1], v.v[4 * h + 2], v.v[4 * h + 3]};
}

template <class T, bool ROWS>
__global__ void __launch_bounds__(512)
k_enc_mxfp4_t(const T* __restrict__ x, int64_t ldx, int64_t rows, int64_t dim, Coded k, Coded kt) {
    constexpr int U = 4;
    __shared__ __align__(1024) uint8_t lds[kTile * kTile * sizeof(T)];
    const Tile2 tile = tile_of<4>(blockIdx.x, (uint32_t)((dim + kTile - 1) / kTile),
                                  (uint32_t)((rows + kTile - 1) / kTile));
    const int64_t r0 = (int64_t)tile.y * kTile, c0 = (int64_t)tile.x * kTile;
    const int t = threadIdx.x;
    const bool whole = r0 + kTile <= rows && c0 + kTile <= dim;
    auto by_rows = [&](auto all) {
        constexpr bool ALL = decltype(all)::value;
        const int64_t col = c0 + 8 * (t & 15);
        Raw8<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r0 + 32 * u + (t >> 4);
            v[u].template load<true>(x + row * ldx + col, ALL ? 8 : row < rows ? dim - col : 0, col > 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r0 + 32 * u + (t >> 4);
            if (!ALL) v[u].settle(row < rows ? dim - col : 0, col > 0);
            if (ROWS) keep_row8<ALL>(v[u], row, col, row < rows, dim, k);
            put_raw8(lds, 32 * u + (t >> 4), 8 * (t & 15), v[u]);
        }
    };
    if (whole) by_rows(std::true_type{});
    else by_rows(std::false_type{});
    __syncthreads();
    // columns 2 pair and 2 pair + 1, rows 32 part + 16 half and on
    const int half = t & 1, pair = t >> 1 & 63, part = t >> 7;
    Columns<T> v;
    v.read(lds, 32 * part + kHalfGroup * half, pair);
    uint32_t m[2];
    v.amax_bits(m);
    const bool group = r0 + 32 * part < rows;  // else: padding, byte 0
    __syncthreads();
    uint8_t* bytes = lds + kTile * 64;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int col = 2 * pair + c;
        const uint32_t byte = mx_byte(pair_of_lanes_max(m[c]));
        const float scale = mx_scale(byte);
        u32x2 w = {v.codes8(0, c, scale), v.codes8(1, c, scale)};
        if (byte == kMxNaN) w = u32x2{0, 0};
        *reinterpret_cast<u32x2*>(lds + col * 64 + ((part ^ ((col >> 2) & 3)) << 4) + 8 * half) = w;
        if (half == 0) bytes[col * 4 + part] = group ? (uint8_t)byte : 0;
    }
    __syncthreads();
    const int to = t >> 2, piece = t & 3;
    if (c0 + to < dim && r0 + 32 * piece < rows)
        *reinterpret_cast<u32x4*>(kt.codes + (c0 + to) * kt.pitch + r0 / 2 + piece * 16) =
            *reinterpret_cast<const u32x4*>(lds + to * 64 + ((piece ^ ((to >> 2) & 3)) << 4));
    if (t < kTile && c0 + t < dim)
        *reinterpret_cast<uint32_t*>(kt.scales + (c0 + t) * kt.spitch + r0 / 32) =
            *reinterpret_cast<const uint32_t*>(bytes + t * 4);
}

// ----------------------------------------------------------------- decode

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int AT>
__device__ __forceinline__ void mx_value_pair(uint32_t word, float scale, float& lo, float& hi) {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, AT);
    lo = v[0];
    hi = v[1];
}

__device__ __forceinline__ float value_or_nan(float v, uint32_t byte) {
    return byte == kMxNaN ? __uint_as_float(0x7FC00000u) : v;
}

// A lane's 8 values of a unit's 128: for bf16 neighbours, 16 bytes of output;
// for fp32 four in each half of the unit, so that a store covers 256 bytes of a
// row without gaps (8192 x 8192: eight neighbours in two stores 105 us).
template <class T>
struct Held8;
template <>
struct Held8<BF16> {
    uint32_t word, byte;
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t unit, int64_t dim) {
        const int64_t col = unit + 8 * (threadIdx.x & 15);
        const bool there = col < dim;
        word = there ? ld_stream_u32(codes + col / 2) : 0u;
        byte = there ? scales[col / 32] : 0u;
    }
    __device__ __forceinline__ void store(BF16* out, int64_t unit, int64_t dim) const {
        const int64_t col = unit + 8 * (threadIdx.x & 15);
        const float scale = mx_scale(byte);
        float v[8];
        mx_value_pair<0>(word, scale, v[0], v[1]);
        mx_value_pair<1>(word, scale, v[2], v[3]);
        mx_value_pair<2>(word, scale, v[4], v[5]);
        mx_value_pair<3>(word, scale, v[6], v[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = value_or_nan(v[i], byte);
        store8(out + col, dim - col, v);
    }
};
template <>
struct Held8<float> {
    uint32_t word[2], byte[2];
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t unit, int64_t dim) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t col = unit + 64 * h + 4 * (threadIdx.x & 15);
            const bool there = col < dim;
            word[h] = there ? ld_stream_u16(codes + col / 2) : 0u;
            byte[h] = there ? scales[col / 32] : 0u;
        }
    }
    __device__ __forceinline__ void store(float* out, int64_t unit, int64_t dim) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t col = unit + 64 * h + 4 * (threadIdx.x & 15), left = dim - col;
            const float scale = mx_scale(byte[h]);
            float v[4];
            mx_value_pair<0>(word[h], scale, v[0], v[1]);
            mx_value_pair<1>(word[h], scale, v[2], v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = value_or_nan(v[i], byte[h]);
            if (left >= 4) {
                const u32x4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                 __float_as_uint(v[3])};
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(out + col));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < left) out[col + i] = v[i];
            }
        }
    }
};

template <class T>
__global__ void __launch_bounds__(256)
k_dec_mxfp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, Sizes z, int64_t pitch,
            int64_t spitch, T* __restrict__ out, int64_t ldo) {
    constexpr int U = kUnroll;
    for (int64_t rt = (int64_t)blockIdx.y * U; rt < z.row_tiles; rt += (int64_t)gridDim.y * U) {
        Held8<T> v[U];
        Place p[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            p[u] = place_of(rt + u, z);
            p[u].col &= ~int64_t(127);
            v[u].load(codes + p[u].row * pitch, scales + p[u].row * spitch, p[u].col, p[u].live ? z.dim : 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) v[u].store(out + p[u].row * ldo, p[u].col, p[u].live ? z.dim : 0);
    }
}

struct Launch {
    Sizes z;
    dim3 grid;
};

Launch launch_of(int64_t rows, int64_t dim) {
    Launch n;
    const int64_t units = (dim + 127) / 128;
    n.z.rows = rows;
    n.z.dim = dim;
    n.z.lx = units >= 16 ? 4 : log2_exact(units);
    n.z.row_tiles = (rows + (16 >> n.z.lx) - 1) >> (4 - n.z.lx);
    const int64_t y = (n.z.row_tiles + kUnroll - 1) / kUnroll;
    n.grid = dim3((unsigned)((units + (1 << n.z.lx) - 1) >> n.z.lx), (unsigned)(y < 65535 ? y : 65535));
    return n;
}

Coded coded(void* codes, void* scales, int64_t dim) {
    return Coded{static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), (dim + 31) / 32 * 16,
                 (dim + 127) / 128 * 4};
}

template <class T>
hipError_t encode(const T* x, int64_t rows, int64_t dim, int64_t ldx, void* codes, void* scales, void* codes_t,
                  void* scales_t, hipStream_t stream) {
    const Coded k = coded(codes, scales, dim), kt = coded(codes_t, scales_t, rows);
    if (!codes_t) {
        const Launch n = launch_of(rows, dim);
        hipLaunchKernelGGL(k_enc_mxfp4<T>, n.grid, dim3(256), 0, stream, x, ldx, n.z, k);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(((dim + kTile - 1) / kTile) * ((rows + kTile - 1) / kTile)));
    if (codes) hipLaunchKernelGGL((k_enc_mxfp4_t<T, true>), grid, dim3(512), 0, stream, x, ldx, rows, dim, k, kt);
    else hipLaunchKernelGGL((k_enc_mxfp4_t<T, false>), grid, dim3(512), 0, stream, x, ldx, rows, dim, k, kt);
    return hipGetLastError();
}

template <class T>
hipError_t decode(const void* codes, const void* scales, int64_t rows, int64_t dim, T* out, int64_t ldo,
                  hipStream_t stream) {
    const Launch n = launch_of(rows, dim);
    hipLaunchKernelGGL(k_dec_mxfp4<T>, n.grid, dim3(256), 0, stream, static_cast<const uint8_t*>(codes),
                       static_cast<const uint8_t*>(scales), n.z, (dim + 31) / 32 * 16, (dim + 127) / 128 * 4, out, ldo);
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
    return bf16 ? decode(codes, scales, rows, dim, static_cast<BF16*>(out), ldo, stream)
                : decode(codes, scales, rows, dim, static_cast<float*>(out), ldo, stream);
}

}  // namespace qc
