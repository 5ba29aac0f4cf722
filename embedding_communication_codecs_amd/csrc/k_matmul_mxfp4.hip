// k_matmul_mxfp4.hip -- C[m][n] (+)= sum over k of A[m][k] B[n][k], both in
// MXFP4 with k contiguous: tokens (A) and weights (B).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 rows x 64 values of each side, a
// lane one group of 32 of a row with its scale byte, and accumulates in fp32.
// The weights are its first operand and the tokens its second, so a lane ends
// up with four times four neighbouring output channels of one token.
//
// The sum may take its groups in any order, and a lane takes four that are
// neighbours, one an instruction: their scale bytes are one word, of which
// each instruction names its byte.
#include "qc_launch.hpp"
#include "qc_lds.hpp"
#include "qc_mx.hpp"

#include <type_traits>

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
    Side a, b;               // tokens, weights
    int64_t pitch, spitch;   // bytes of a row: codes, scales
    int64_t ldc;
    int stages_per_split;    // stages of 128 bytes of codes; blockIdx.y: the split
    int64_t split_stride;    // elements of c between two splits' sums
};

__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// BYTE: which of the scale words' bytes.
template <int BYTE>
__device__ __forceinline__ f32x16 mfma32(i32x4 b, i32x4 a, f32x16 c, int sb, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(b), operand(a), c, 4, 4, BYTE, sb, BYTE, sa);
}
__device__ __forceinline__ f32x16 mfma32(int byte, i32x4 b, i32x4 a, f32x16 c, int sb, int sa) {
    switch (byte) {  // known where the loops are unrolled
        case 0: return mfma32<0>(b, a, c, sb, sa);
        case 1: return mfma32<1>(b, a, c, sb, sa);
        case 2: return mfma32<2>(b, a, c, sb, sa);
        default: return mfma32<3>(b, a, c, sb, sa);
    }
}
template <int BYTE>
__device__ __forceinline__ f32x4 mfma16(i32x4 b, i32x4 a, f32x4 c, int sb, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b), operand(a), c, 4, 4, BYTE, sb, BYTE, sa);
}
__device__ __forceinline__ f32x4 mfma16(int byte, i32x4 b, i32x4 a, f32x4 c, int sb, int sa) {
    switch (byte) {
        case 0: return mfma16<0>(b, a, c, sb, sa);
        case 1: return mfma16<1>(b, a, c, sb, sa);
        case 2: return mfma16<2>(b, a, c, sb, sa);
        default: return mfma16<3>(b, a, c, sb, sa);
    }
}

__device__ __forceinline__ u32x2 packed4(const BF16*, const float (&v)[4]) {
    return u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}
__device__ __forceinline__ f32x4 packed4(const float*, const float (&v)[4]) { return f32x4{v[0], v[1], v[2], v[3]}; }

// c, or c plus what is there.
template <bool ADD>
__device__ __forceinline__ void put_result(float* p, float v) { *p = ADD ? *p + v : v; }
template <bool ADD>
__device__ __forceinline__ void put_result(BF16* p, float v) {
    static_assert(!ADD, "sums are added to in fp32 only");
    put(p, v);
}

// ------------------------------------------------------- pipelined tiles
// One block computes BN channels x BM tokens with WN x WM waves, in stages of
// 128 bytes of codes a row (256 values, 8 groups), NB of them in LDS.
//
// Codes: 8 rows x 128 bytes a load; the eight 16-byte pieces of a row lie
// permuted, so that the fragment reads are free of bank conflicts (16
// neighbouring rows of one piece differ modulo 256 bytes).
// Scales: 8 bytes a row and stage would be a load that touches 32 rows for
// 256 bytes; they are fetched 32 bytes a row, for four stages (a chunk) at a
// time, a quarter of the tile's rows with each stage.
constexpr int kStage = 128, kChunk = 4, kScaleBytes = 8 * kChunk;

__device__ __forceinline__ int piece_slot(int row, int piece) { return piece ^ ((row >> 1) & 7); }

// Rows [row0, row0 + ROWS) of a matrix's codes, `len` bytes of each.  Rows past
// the matrix repeat its last row (their results are not stored) and pieces past
// a row's end its last piece (made zeros before use), so every address is
// inside the matrix.
template <int ROWS, int NW>
struct Loader {
    static constexpr int N = ROWS / 8 / NW;  // loads a wave
    static_assert(N >= 1 && N * 8 * NW == ROWS, "every wave loads alike");
    int off[N];
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ void init(const uint8_t* codes, int64_t pitch, int64_t row0, int64_t rows, int len,
                                         int wave) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = min(row(wave, i), last) * (int)pitch + piece(wave, i) * 16;
        rsrc = buffer_of(codes + row0 * pitch, last * (int)pitch + len);
    }
    __device__ __forceinline__ static int row(int wave, int i) { return (wave * N + i) * 8 + lane_id() / 8; }
    __device__ __forceinline__ static int piece(int wave, int i) { return piece_slot(row(wave, i), lane_id() % 8); }
    // load `i` of N of stage s.  WHOLE: the rows reach the stage's end.
    template <bool WHOLE>
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, int s, int len) const {
        const int over = WHOLE ? 0 : max(s * kStage + piece(wave, i) * 16 - (len - 16), 0);
        load_lds16(rsrc, lds + (wave * N + i) * 1024, off[i] - over, s * kStage);
    }
};

// Their scales: blocks of 32 rows x one chunk, 1 KiB of LDS, a row's two pieces
// in turn so that neighbouring eights of rows lie in different banks.
__device__ __forceinline__ int scale_piece(int row, int piece) { return piece ^ ((row >> 3) & 1); }

struct ScaleLoader {
    __amdgpu_buffer_rsrc_t rsrc;
    int last, pitch;
    __device__ __forceinline__ void init(const uint8_t* scales, int64_t spitch, int64_t row0, int64_t rows, int span,
                                         int len) {
        const int64_t left = rows - 1 - row0;
        last = left < span - 1 ? (int)left : span - 1;
        pitch = (int)spitch;
        rsrc = buffer_of(scales + row0 * spitch, last * pitch + len);
    }
    // Rows [first, first + 32) of chunk c to `lds`; `len` bytes of a row exist.
    // FAST: they are at least one piece, and either whole pieces or reach the
    // chunk's end.  What lies past them repeats others and is not used.
    template <bool FAST>
    __device__ __forceinline__ void load(int first, int c, int len, uint32_t lds) const {
        const int l = lane_id();
        if constexpr (FAST) {
            const int r = l >> 1, at = min(c * kScaleBytes + scale_piece(r, l & 1) * 16, len - 16);
            load_lds16(rsrc, lds, min(first + r, last) * pitch + at, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int slot = e * 16 + (l >> 2), r = slot >> 1;
                const int at = c * kScaleBytes + scale_piece(r, slot & 1) * 16 + (l & 3) * 4;
                load_lds4(rsrc, lds + e * 256, min(first + r, last) * pitch + min(at, len - 4), 0);
            }
        }
    }
};

// A wave reads its fragments ahead of their use, into the next stage too; the
// wait for that stage, and the only barrier, stand where the last fragments of
// this one have been read, and the fragments already in registers keep the
// matrix cores busy across it.  The loads of the stage NB further on follow at
// once, over the one just left.  A stage has no branch: the compiler would move
// matrix instructions across it, and their operands would fill the registers.
// So loads are issued past the end too (they repeat the last pieces), and where
// a tile has fewer blocks of scales a stage than waves, several load the same.
template <class T, bool ADD, int BN, int BM, int WN, int WM, int NB>
__global__ void __launch_bounds__(WN * WM * WAVE)
k_mm_mx_pipe(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM;
    constexpr int FN = BN / WN / 32, FM = BM / WM / 32;
    constexpr int AHEAD = FN >= 4 ? 2 : 1;          // weight fragments read ahead (of a ring)
    constexpr int RING = FN >= 4 ? 4 : 2;
    constexpr int KK = 4, STEPS = KK * FN;          // a step: one weight fragment
    constexpr int H = (FN + 1) / 2, TURN = STEPS - H;  // the barrier's step
    constexpr int TB = BN * kStage, STAGE = (BN + BM) * kStage;  // weights first, then tokens
    constexpr int NC = NB == 2 ? 2 : 3, SBLOCKS = (BN + BM) / 128;  // chunks in LDS; blocks of scales a stage
    // a stage's last read comes before the barrier, the next one's first after it
    static_assert(FM >= 1 && STEPS - 1 - AHEAD <= TURN && STEPS - AHEAD >= TURN && SBLOCKS * 128 == BN + BM, "tile");
    static_assert(NB * STAGE + NC * (BN + BM) * kScaleBytes <= 160 * 1024 && NB >= 2 && NB <= 4, "LDS");
    __shared__ __align__(1024) uint8_t lds[NB * STAGE + NC * (BN + BM) * kScaleBytes];

    const uint32_t tn = (uint32_t)((g.b.rows + BN - 1) / BN), tm = (uint32_t)((g.a.rows + BM - 1) / BM);
    const Tile2 tile = tile_of<4>(blockIdx.x, tn, tm);
    const int64_t n0 = (int64_t)tile.x * BN, m0 = (int64_t)tile.y * BM;
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wm = w / WN;
    const int l = lane_id(), half = l >> 5;
    // this split's part of a row
    const int first = (int)blockIdx.y * g.stages_per_split;
    const int len = min((int)g.pitch - first * kStage, g.stages_per_split * kStage);
    const int slen = (int)g.spitch - first * 8;
    const int stages = (len + kStage - 1) / kStage, whole = len / kStage;
    Loader<BN, NW> lb;
    Loader<BM, NW> la;
    constexpr int LOADS = lb.N + la.N;
    lb.init(g.b.codes + first * kStage, g.pitch, n0, g.b.rows, len, w);
    la.init(g.a.codes + first * kStage, g.pitch, m0, g.a.rows, len, w);
    ScaleLoader xb, xa;
    xb.init(g.b.scales + first * 8, g.spitch, n0, g.b.rows, BN, slen);
    xa.init(g.a.scales + first * 8, g.spitch, m0, g.a.rows, BM, slen);

    const uint32_t lds0 = lds_addr(lds);
    auto fetch_part = [&](auto fast, int part, int buf, int s) {  // one of LOADS
        constexpr bool FAST = decltype(fast)::value;
        if (part < lb.N) lb.template load<FAST>(part, lds0 + buf * STAGE, w, s, len);
        else la.template load<FAST>(part - lb.N, lds0 + buf * STAGE + TB, w, s, len);
    };
    auto fetch_scales = [&](auto fast, int chunk, int quarter) {
        const int block = quarter * SBLOCKS + w % SBLOCKS;
        const bool weights = block * 32 < BN;
        const ScaleLoader x = {weights ? xb.rsrc : xa.rsrc, weights ? xb.last : xa.last, xb.pitch};
        x.template load<decltype(fast)::value>(block * 32 - (weights ? 0 : BN), chunk, slen,
                                               lds0 + NB * STAGE + (chunk % NC) * ((BN + BM) * kScaleBytes) +
                                                   block * 1024);
    };

    // fragments: row l % 32, piece half * 4 + kk (an xor of kk * 16 in the address)
    const int frag = (l & 31) * kStage + (piece_slot(l & 31, half * 4) << 4);
    const int rb = wn * FN * 32 * kStage + frag, ra = TB + wm * FM * 32 * kStage + frag;
    auto read_b = [&](auto fast, int buf, int q, int s) {
        i32x4 v = *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (rb ^ (q / FN * 16)) + q % FN * (32 * kStage));
        // the weights' pieces past a row's end become zeros (one side is enough)
        if (!decltype(fast)::value && s * kStage + (half * 4 + q / FN) * 16 >= len) v = i32x4{0, 0, 0, 0};
        return v;
    };
    auto read_a = [&](int buf, int kk, int j) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (ra ^ (kk * 16)) + j * (32 * kStage));
    };
    int sb[FN], sa[FM];
    auto read_scales = [&](int s, int (&nb)[FN], int (&na)[FM]) {
        const uint8_t* at = lds + NB * STAGE + (s / kChunk % NC) * ((BN + BM) * kScaleBytes) + (l & 31) * kScaleBytes +
                            (scale_piece(l & 31, (s >> 1) & 1) << 4) + ((s & 1) << 3) + (half << 2);
        const bool there = s * 8 + half * 4 < slen;  // words past a row's end are another row's
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int v = *reinterpret_cast<const int*>(at + (wn * FN + i) * 1024);
            nb[i] = there ? v : 0;
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int v = *reinterpret_cast<const int*>(at + BN * kScaleBytes + (wm * FM + j) * 1024);
            na[j] = there ? v : 0;
        }
    };

    f32x16 acc[FN][FM] = {};
    i32x4 fb[RING], fa[2][FM];
    // Stage s in buffer `buf`, the next one in `next`.  Fast: stages up to s +
    // NB exist and are whole.
    auto stage = [&](int buf, int next, auto fast, int s) {
        int nb[FN], na[FM];
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int kk = q / FN, i = q % FN;
            if (q + AHEAD < STEPS) fb[(q + AHEAD) % RING] = read_b(fast, buf, q + AHEAD, s);
            if (q == TURN) {
                lds_landed_but<(NB - 2) * LOADS>();
                fetch_scales(fast, (s + NB - 1) / kChunk + 1, (s + NB - 1) % kChunk);
                read_scales(s + 1, nb, na);
            }
            if (q + AHEAD >= STEPS) fb[(q + AHEAD) % RING] = read_b(fast, next, q + AHEAD - STEPS, s + 1);
            if (i >= FN - H) {
                // this step's share of the token fragments and of the loads
                const int part = i - (FN - H);
#pragma unroll
                for (int e = part * FM / H; e < (part + 1) * FM / H; ++e)
                    fa[(kk + 1) & 1][e] = kk + 1 < KK ? read_a(buf, kk + 1, e) : read_a(next, 0, e);
                if (kk + 1 == KK) {
#pragma unroll
                    for (int d = part * LOADS / H; d < (part + 1) * LOADS / H; ++d) fetch_part(fast, d, buf, s + NB);
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = mfma32(kk, fb[q % RING], fa[kk & 1][j], acc[i][j], sb[i], sa[j]);
            __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) sb[i] = nb[i];
#pragma unroll
        for (int j = 0; j < FM; ++j) sa[j] = na[j];
    };

#pragma unroll
    for (int x = 0; x < kChunk + NB - 1; ++x) fetch_scales(std::false_type{}, x / kChunk, x % kChunk);
#pragma unroll
    for (int s = 0; s < NB; ++s) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) fetch_part(std::false_type{}, part, s, s);
    }
    lds_landed_but<(NB - 1) * LOADS>();
    read_scales(0, sb, sa);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[0][j] = read_a(0, 0, j);
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) fb[q] = read_b(std::false_type{}, 0, q, 0);
    // fast stages: where rows of scales end inside a piece, those whose chunks are whole
    const int fast_end = min(whole, slen % 16 == 0 ? whole : slen / kScaleBytes * kChunk - kChunk + 1);
    int s = 0;
    for (; s + 2 * NB - 1 < fast_end; s += NB) {
#pragma unroll
        for (int u = 0; u < NB; ++u) stage(u, (u + 1) % NB, std::true_type{}, s + u);
    }
#pragma unroll 1
    for (; s < stages; ++s) stage(s % NB, (s + 1) % NB, std::false_type{}, s);

    // 32 tokens at a time through the wave's part of LDS, so that a store takes
    // whole 16-byte pieces of a few rows of C.  Piece p of row r in slot p ^ r.
    constexpr int COLS = FN * 32, RB = COLS * (int)sizeof(T), PR = RB / 16, E = 16 / (int)sizeof(T);
    static_assert((PR & (PR - 1)) == 0 && PR <= WAVE && NW * 32 * RB <= NB * STAGE, "a wave's part of LDS");
    lds_landed();  // every wave has read its last fragments, and no load is on its way
    uint8_t* own = lds + w * (32 * RB);
    c += (int64_t)blockIdx.y * g.split_stride;
    const bool inside = n0 + BN <= g.b.rows && m0 + BM <= g.a.rows;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
                const int at = (i * 32 + q * 8 + 4 * half) * (int)sizeof(T), r = l & 31;
                const auto four = packed4(c, v);
                *reinterpret_cast<std::remove_const_t<decltype(four)>*>(
                    own + r * RB + (((at >> 4) ^ (r & (PR - 1))) << 4) + (at & 15)) = four;
            }
        }
        wave_lds_sync();
        const int64_t row0 = m0 + (wm * FM + j) * 32, col0 = n0 + wn * COLS;
#pragma unroll
        for (int q = 0; q < RB / 32; ++q) {
            const int r = (q * WAVE + l) / PR, p = (q * WAVE + l) % PR;
            const uint8_t* from = own + r * RB + ((p ^ (r & (PR - 1))) << 4);
            const int64_t row = row0 + r, col = col0 + p * E, left = inside || row < g.a.rows ? g.b.rows - col : 0;
            T* to = c + row * g.ldc + col;
            if (inside || left >= E) {
                u32x4 v = *reinterpret_cast<const u32x4*>(from);
                if constexpr (ADD) {
                    const u32x4 old = *reinterpret_cast<const u32x4_a2*>(to);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = __float_as_uint(__uint_as_float(old[e]) + __uint_as_float(v[e]));
                }
                *reinterpret_cast<u32x4_a2*>(to) = v;
            } else {
                for (int e = 0; e < E; ++e)
                    if (e < left) put_result<ADD>(to + e, to_f32(reinterpret_cast<const T*>(from)[e]));
            }
        }
        wave_lds_sync();
    }
}

template <class T, bool ADD, int BN, int BM, int WN, int WM, int NB>
hipError_t launch_pipe(const Args& g, int splits, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.b.rows + BN - 1) / BN) * ((g.a.rows + BM - 1) / BM);
    hipLaunchKernelGGL((k_mm_mx_pipe<T, ADD, BN, BM, WN, WM, NB>), dim3((unsigned)tiles, splits), dim3(WN * WM * WAVE),
                       0, stream, g, c);
    return hipGetLastError();
}

// ------------------------------------------------------------- few tokens
// One block: NT * 16 channels x MT * 16 tokens, k split over WS waves in
// slabs of 256 bytes of codes (512 values), joined through LDS.  A wave loads
// the rows of its slab into a part of LDS of its own (no barrier until the
// waves join), up to NB slabs at a time, as 4 rows x 256 bytes a load, and
// their scales as 16 rows x 16 bytes.
constexpr int kSlab = 256;

template <int ROWS>
struct SlabLoader {
    static constexpr int N = ROWS / 4 + ROWS / 16;  // loads of a slab
    static constexpr int BYTES = ROWS * (kSlab + 16);
    int off[ROWS / 4], soff[ROWS / 16];
    __amdgpu_buffer_rsrc_t rsrc, srsrc;
    __device__ __forceinline__ static int piece(int i) { return (lane_id() % 16) ^ ((i * 4 + lane_id() / 16) & 15); }
    __device__ __forceinline__ void init(const Side& s, int64_t row0, int64_t pitch, int64_t spitch) {
        const int64_t left = s.rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
#pragma unroll
        for (int i = 0; i < ROWS / 4; ++i)
            off[i] = min(i * 4 + lane_id() / 16, last) * (int)pitch + piece(i) * 16;
#pragma unroll
        for (int i = 0; i < ROWS / 16; ++i)
            soff[i] = min(i * 16 + lane_id() / 4, last) * (int)spitch + (lane_id() % 4) * 4;
        rsrc = buffer_of(s.codes + row0 * pitch, (last + 1) * (int)pitch);
        srsrc = buffer_of(s.scales + row0 * spitch, (last + 1) * (int)spitch);
    }
    // what lies past a row's end repeats its last piece, or word
    __device__ __forceinline__ void load(int slab, uint32_t lds, int pitch, int spitch) const {
#pragma unroll
        for (int i = 0; i < ROWS / 4; ++i)
            load_lds16(rsrc, lds + i * 1024, off[i] - max(slab * kSlab + piece(i) * 16 - (pitch - 16), 0), slab * kSlab);
#pragma unroll
        for (int i = 0; i < ROWS / 16; ++i)
            load_lds4(srsrc, lds + ROWS * kSlab + i * 256,
                      soff[i] - max(slab * 16 + (lane_id() % 4) * 4 - (spitch - 4), 0), slab * 16);
    }
};

template <class T, bool ADD, int NT, int MT, int WS, int NB>
__global__ void __launch_bounds__(WS * WAVE)
k_mm_mx_few(Args g, T* __restrict__ c) {
    typedef SlabLoader<NT * 16> LB;
    typedef SlabLoader<MT * 16> LA;
    constexpr int SLAB = LB::BYTES + LA::BYTES, LOADS = LB::N + LA::N;
    constexpr int OWN = NB * SLAB > NT * MT * 1024 ? NB * SLAB : NT * MT * 1024;  // a wave's LDS: slabs, then sums
    static_assert(WS * OWN <= 160 * 1024, "LDS");
    __shared__ __align__(1024) uint8_t lds[WS * OWN];
    const int l = lane_id(), quad = l >> 4, w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t tn = (uint32_t)((g.b.rows + NT * 16 - 1) / (NT * 16));
    const int64_t n0 = (int64_t)(blockIdx.x % tn) * (NT * 16), m0 = (int64_t)(blockIdx.x / tn) * (MT * 16);
    const int pitch = (int)g.pitch, spitch = (int)g.spitch;
    LB lb;
    LA la;
    lb.init(g.b, n0, g.pitch, g.spitch);
    la.init(g.a, m0, g.pitch, g.spitch);
    uint8_t* own = lds + w * OWN;
    auto fetch = [&](int slab, int buf) {
        const uint32_t at = lds_addr(own) + buf * SLAB;
        lb.load(slab, at, pitch, spitch);
        la.load(slab, at + LB::BYTES, pitch, spitch);
    };

    f32x4 acc[NT][MT] = {};
    const int slabs = (pitch + kSlab - 1) / kSlab;
    const int mine = (slabs - w + WS - 1) / WS;  // slabs w, w + WS, ...
#pragma unroll
    for (int b = 0; b < NB; ++b)
        if (b < mine) fetch(w + b * WS, b);
    for (int it = 0; it < mine; ++it) {
        const int slab = w + it * WS, buf = NB == 1 ? 0 : it % NB;
        if (NB > 1 && it + NB <= mine) asm volatile("s_waitcnt vmcnt(%0)" : : "n"((NB - 1) * LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        const uint8_t* at = own + buf * SLAB;
        const bool there = slab * 16 + quad * 4 < spitch;
        int sb[NT], sa[MT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int v = *reinterpret_cast<const int*>(at + NT * 16 * kSlab + i * 256 + (l & 15) * 16 + quad * 4);
            sb[i] = there ? v : 0;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int v = *reinterpret_cast<const int*>(at + LB::BYTES + MT * 16 * kSlab + j * 256 + (l & 15) * 16 +
                                                        quad * 4);
            sa[j] = there ? v : 0;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int piece = quad * 4 + kk, slot = (piece ^ (l & 15)) << 4;
            i32x4 fb[NT], fa[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                fb[i] = *reinterpret_cast<const i32x4*>(at + (i * 16 + (l & 15)) * kSlab + slot);
                if (slab * kSlab + piece * 16 >= pitch) fb[i] = i32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
                fa[j] = *reinterpret_cast<const i32x4*>(at + LB::BYTES + (j * 16 + (l & 15)) * kSlab + slot);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = mfma16(kk, fb[i], fa[j], acc[i][j], sb[i], sa[j]);
        }
        if (it + NB < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // this slab has been read
            fetch(slab + NB * WS, buf);
        }
    }

    // all of a wave's loads have landed and been read; its part of LDS takes its sums
    f32x4* sums = reinterpret_cast<f32x4*>(own);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) sums[(i * MT + j) * WAVE + l] = acc[i][j];
    __syncthreads();
    for (int f = w; f < NT * MT; f += WS) {
        f32x4 sum = {};
#pragma unroll
        for (int s = 0; s < WS; ++s) sum += *reinterpret_cast<const f32x4*>(lds + s * OWN + (f * WAVE + l) * 16);
        const int64_t row = m0 + (f % MT) * 16 + (l & 15);
        const int64_t col = n0 + (f / MT) * 16 + 4 * quad;
        if (row < g.a.rows) {
            T* to = c + row * g.ldc + col;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < g.b.rows) put_result<ADD>(to + e, sum[e]);
        }
    }
}

template <class T, bool ADD, int NT, int MT, int WS, int NB>
hipError_t launch_few(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.b.rows + NT * 16 - 1) / (NT * 16)) * ((g.a.rows + MT * 16 - 1) / (MT * 16));
    hipLaunchKernelGGL((k_mm_mx_few<T, ADD, NT, MT, WS, NB>), dim3((unsigned)tiles), dim3(WS * WAVE), 0, stream, g, c);
    return hipGetLastError();
}

// ------------------------------------------------------------------ choice
// Placeholder rule: few tokens by 16 x 16 to 32 x 64, else by pipelined tiles.
template <class T, bool ADD>
hipError_t launch_shape(int shape, const Args& g, int splits, T* c, hipStream_t stream) {
    switch (shape) {
        case 0: return launch_few<T, ADD, 1, 1, 8, 2>(g, c, stream);
        case 1: return launch_few<T, ADD, 2, 1, 6, 2>(g, c, stream);
        case 2: return launch_few<T, ADD, 2, 2, 8, 1>(g, c, stream);
        case 3: return launch_few<T, ADD, 2, 4, 6, 1>(g, c, stream);
        case 4: return launch_pipe<T, ADD, 64, 64, 1, 2, 4>(g, splits, c, stream);
        case 5: return launch_pipe<T, ADD, 128, 128, 1, 4, 4>(g, splits, c, stream);
        case 6: return launch_pipe<T, ADD, 128, 256, 1, 4, 2>(g, splits, c, stream);
        case 7: return launch_pipe<T, ADD, 256, 256, 2, 4, 2>(g, splits, c, stream);
        default: return launch_pipe<T, ADD, 256, 256, 2, 2, 2>(g, splits, c, stream);
    }
}

int shape_of(int64_t m, int64_t n) {
    if (m <= 16) return 0;
    if (m <= 32) return 2;
    if (m <= 64) return 3;
    return ((m + 255) / 256) * ((n + 255) / 256) >= 200 ? 7 : 5;
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
    const int64_t pitch = (k + 31) / 32 * 16;
    const Args g{{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales), m},
                 {static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales), n},
                 pitch, (k + 127) / 128 * 4, ldc, (int)((pitch + kStage - 1) / kStage), 0};
    const int shape = shape_of(m, n);
    if (bf16) return launch_shape<BF16, false>(shape, g, 1, static_cast<BF16*>(c), stream);
    return accumulate ? launch_shape<float, true>(shape, g, 1, static_cast<float*>(c), stream)
                      : launch_shape<float, false>(shape, g, 1, static_cast<float*>(c), stream);
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
