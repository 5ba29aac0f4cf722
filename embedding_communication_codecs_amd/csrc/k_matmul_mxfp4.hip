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

constexpr int kUnits = 256;  // compute units

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
                                         int wave, int lane) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = min(row(wave, i, lane), last) * (int)pitch + piece(wave, i, lane) * 16;
        rsrc = buffer_of(codes + row0 * pitch, last * (int)pitch + len);
    }
    __device__ __forceinline__ static int row(int wave, int i, int lane) { return (wave * N + i) * 8 + lane / 8; }
    __device__ __forceinline__ static int piece(int wave, int i, int lane) {
        return piece_slot(row(wave, i, lane), lane % 8);
    }
    // load `i` of N of stage s.  WHOLE: the rows reach the stage's end.  Where they
    // may not, the stage is part of a lane's own offset: beside it, what brings a
    // piece of a stage past the end back to the row's last one would make that
    // offset negative, which buffer addressing takes for one past the descriptor.
    template <bool WHOLE>
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, int s, int len) const {
        const uint32_t to = lds + (wave * N + i) * 1024;
        if constexpr (WHOLE) load_lds16(rsrc, to, off[i], s * kStage);
        else load_lds16(rsrc, to, off[i] + min(s * kStage, len - 16 - piece(wave, i, lane_id()) * 16), 0);
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
    // Rows [first, first + 32) of chunk c to `lds`, by the waves whose mask is not
    // 0; `len` bytes of a row exist.
    // FAST: they are at least one piece, and either whole pieces or reach the
    // chunk's end.  What lies past them repeats others and is not used.
    template <bool FAST>
    __device__ __forceinline__ void load(int mask, int first, int c, int len, uint32_t lds) const {
        const int l = lane_id();
        if constexpr (FAST) {
            const int r = l >> 1, at = min(c * kScaleBytes + scale_piece(r, l & 1) * 16, len - 16);
            load_lds16_if(mask, rsrc, lds, min(first + r, last) * pitch + at);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int slot = e * 16 + (l >> 2), r = slot >> 1;
                const int at = c * kScaleBytes + scale_piece(r, slot & 1) * 16 + (l & 3) * 4;
                load_lds4_if(mask, rsrc, lds + e * 256, min(first + r, last) * pitch + min(at, len - 4));
            }
        }
    }
};

// WN x WM waves share the tile, and KW (1 or 2) of them each one's part: two
// take the four instructions' worth of k of a stage between them, so that a wave
// of a small tile has two fragments of either side to multiply, and join their
// sums at the end.  A wave reads the fragments of its next step while it
// multiplies those of this one.  Before the last step of a stage has its turn,
// all of the stage's fragments have been read: there stand the wait for the next
// stage and the only barrier, and the matrix cores work on across it. The loads
// of the stage NB further on follow, over the one just left: SOON of them at
// once, the others with the steps of the next stage, as many at a time would
// hold up the wave (16384 x 8192 x 8192: 487 us against 512).  The next stage's
// scales, whose chunk was complete a stage ago, are read a step before the turn:
// 32 bytes a row put four rows in a bank, a read takes 8 cycles of LDS, and six
// of them from each wave, all at once behind the barrier, were ahead of the
// fragments there (510 us against 520).  A stage has no branch: the compiler
// would move matrix instructions across it, and their operands would fill the
// registers.  So loads are issued past the end too (they repeat the last
// pieces), and those of the scales by fewer waves than there are with an empty
// mask in the others.
//
// The two largest tiles, of whose blocks a compute unit holds one, go on to
// further tiles (LOOP): the scales and the first stage of the next one are on
// their way while the results of this one leave through the other stage's
// buffer (16384 x 8192 x 8192 501 us against 508 with a block for each tile,
// with tiles of 128 x 256 646 against 661).  More would need their stores out of
// the way of the waits for loads, which count both in one order.
template <class T, bool ADD, int BN, int BM, int WN, int WM, int KW, int NB>
__global__ void __launch_bounds__(WN * WM * KW * WAVE)
k_mm_mx_pipe(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM * KW, STEPS = 4 / KW;
    constexpr bool LOOP = KW == 1 && NB == 2;
    constexpr int FN = BN / WN / 32, FM = BM / WM / 32;
    constexpr int TB = BN * kStage, STAGE = (BN + BM) * kStage;  // weights first, then tokens
    constexpr int NC = NB == 2 ? 2 : 3;                          // chunks in LDS
    constexpr int BLOCKS = (BN + BM) / 32, SBLOCKS = (BLOCKS + 3) / 4;  // of scales: a chunk's, a stage's
    static_assert(FN >= 1 && FM % KW == 0 && FN * WN * 32 == BN && FM * WM * 32 == BM && STEPS % 2 == 0, "tile");
    static_assert(NB * STAGE + NC * BLOCKS * 1024 <= 160 * 1024 && NB >= 2 && NB <= 4, "LDS");
    __shared__ __align__(1024) uint8_t lds[NB * STAGE + NC * BLOCKS * 1024];

    // results, 32 tokens x FS * 32 columns at a time: bytes of a row, its 16-byte pieces, elements of one, stores
    constexpr int OM = FM / KW, SPACE = (LOOP ? 1 : NB) * STAGE;
    constexpr int FS = NW * 32 * FN * 32 * (int)sizeof(T) <= SPACE ? FN : FN / 2;
    constexpr int RB = FS * 32 * (int)sizeof(T), PR = RB / 16, E = 16 / (int)sizeof(T), STORES = RB / 32;
    static_assert((PR & (PR - 1)) == 0 && PR <= WAVE && NW * 32 * RB <= SPACE && FN % FS == 0, "a wave's part of LDS");

    const uint32_t tn = (uint32_t)((g.b.rows + BN - 1) / BN), tm = (uint32_t)((g.a.rows + BM - 1) / BM);
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wk = w % KW, wn = w / KW % WN, wm = w / KW / WN;
    const int l = lane_id(), half = l >> 5;
    // this split's part of a row
    const int first = (int)blockIdx.y * g.stages_per_split;
    c += (int64_t)blockIdx.y * g.split_stride;
    const int len = min((int)g.pitch - first * kStage, g.stages_per_split * kStage);
    const int slen = (int)g.spitch - first * 8;
    const int stages = (len + kStage - 1) / kStage, whole = len / kStage;
    Loader<BN, NW> lb;
    Loader<BM, NW> la;
    constexpr int LOADS = lb.N + la.N, SOON = LOADS / 4;
    constexpr int SLOTS = (STEPS - 1) * FN, LATER = (LOADS - SOON + SLOTS - 1) / SLOTS;  // of the others at a time
    ScaleLoader xb, xa;
    int64_t n0, m0;
    auto go_to = [&](uint32_t id) {
        const Tile2 tile = tile_of<4>(id, tn, tm);
        n0 = (int64_t)tile.x * BN;
        m0 = (int64_t)tile.y * BM;
        int lane = lane_id();  // opaque: what follows from it is not kept over the loop of stages
        asm volatile("" : "+v"(lane));
        lb.init(g.b.codes + first * kStage, g.pitch, n0, g.b.rows, len, w, lane);
        la.init(g.a.codes + first * kStage, g.pitch, m0, g.a.rows, len, w, lane);
        xb.init(g.b.scales + first * 8, g.spitch, n0, g.b.rows, BN, slen);
        xa.init(g.a.scales + first * 8, g.spitch, m0, g.a.rows, BM, slen);
    };

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
    auto fetch_part = [&](auto fast, int part, int buf, int s) {  // one of LOADS
        constexpr bool FAST = decltype(fast)::value;
        if (part < lb.N) lb.template load<FAST>(part, lds0 + buf * STAGE, w, s, len);
        else la.template load<FAST>(part - lb.N, lds0 + buf * STAGE + TB, w, s, len);
    };
    auto fetch_scales = [&](auto fast, int chunk, int quarter) {
        const int block = min(quarter * SBLOCKS + w % SBLOCKS, BLOCKS - 1);
        const int mask = w < SBLOCKS ? -1 : 0;
        const bool weights = block * 32 < BN;
        const ScaleLoader x = {weights ? xb.rsrc : xa.rsrc, weights ? xb.last : xa.last, xb.pitch};
        x.template load<decltype(fast)::value>(mask, block * 32 - (weights ? 0 : BN), chunk, slen,
                                               lds0 + NB * STAGE + (chunk % NC * BLOCKS + block) * 1024);
    };

    // fragments: row l % 32, piece half * 4 + kk (an xor of kk * 16 in the address)
    const int frag = (l & 31) * kStage + (piece_slot(l & 31, half * 4) << 4);
    const int rb = wn * FN * 32 * kStage + frag, ra = TB + wm * FM * 32 * kStage + frag;
    auto read_b = [&](auto fast, int buf, int kk, int i, int s) {
        i32x4 v = *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (rb ^ (kk * 16)) + i * (32 * kStage));
        // the weights' pieces past a row's end become zeros (one side is enough)
        if (!decltype(fast)::value && s * kStage + (half * 4 + kk) * 16 >= len) v = i32x4{0, 0, 0, 0};
        return v;
    };
    auto read_a = [&](int buf, int kk, int j) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (ra ^ (kk * 16)) + j * (32 * kStage));
    };
    int sb[FN], sa[FM];
    auto read_scales = [&](int s, int (&nb)[FN], int (&na)[FM]) {
        const uint8_t* at = lds + NB * STAGE + (s / kChunk % NC) * (BLOCKS * 1024) + (l & 31) * kScaleBytes +
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
    // a wave's own instructions of a stage: with KW > 1 the byte of the scale
    // words that they name depends on the wave, so it is brought down
    auto mine = [&](int (&x)[FN], int (&y)[FM]) {
        if constexpr (KW > 1) {
#pragma unroll
            for (int i = 0; i < FN; ++i) x[i] = (int)((uint32_t)x[i] >> (8 * STEPS * wk));
#pragma unroll
            for (int j = 0; j < FM; ++j) y[j] = (int)((uint32_t)y[j] >> (8 * STEPS * wk));
        }
    };

    f32x16 acc[FN][FM];
    i32x4 fb[2][FN], fa[2][FM];
    // Stage s in buffer `buf`, the next one in `next`.  Fast: stages up to s +
    // NB exist and are whole.
    auto stage = [&](int buf, int next, auto fast, int s) {
        int nb[FN], na[FM];
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
            const bool turn = t + 1 == STEPS;
            if (turn) {
                lds_landed_but<(NB - 2) * LOADS>();
                fetch_scales(fast, (s + NB) / kChunk + 1, (s + NB) % kChunk);
            }
            if (t + 2 == STEPS) read_scales(s + 1, nb, na);
            // the next step's fragments
            const int kk = turn ? wk * STEPS : wk * STEPS + t + 1, at = turn ? next : buf, ns = turn ? s + 1 : s;
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[(t + 1) & 1][j] = read_a(at, kk, j);
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                fb[(t + 1) & 1][i] = read_b(fast, at, kk, i, ns);
                if (turn) {
#pragma unroll
                    for (int d = i * SOON / FN; d < (i + 1) * SOON / FN; ++d) fetch_part(fast, d, buf, s + NB);
                } else {
                    // the rest of the stage before's loads
#pragma unroll
                    for (int d = SOON + (t * FN + i) * LATER; d < min(LOADS, SOON + (t * FN + i + 1) * LATER); ++d)
                        fetch_part(fast, d, (buf + NB - 1) % NB, s + NB - 1);
                }
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = mfma32(t, fb[t & 1][i], fa[t & 1][j], acc[i][j], sb[i], sa[j]);
                __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
            }
        }
        mine(nb, na);
#pragma unroll
        for (int i = 0; i < FN; ++i) sb[i] = nb[i];
#pragma unroll
        for (int j = 0; j < FM; ++j) sa[j] = na[j];
    };

    // A tile's first loads: scales and all stages but the last of NB.  Stage s
    // lies in buffer (s + 1) % NB, so that these leave buffer 0 alone.
    auto begin = [&]() {
#pragma unroll
        for (int x = 0; x < kChunk + NB; ++x) fetch_scales(std::false_type{}, x / kChunk, x % kChunk);
#pragma unroll
        for (int s = 0; s + 1 < NB; ++s) {
#pragma unroll
            for (int part = 0; part < LOADS; ++part) fetch_part(std::false_type{}, part, s + 1, s);
        }
    };
    go_to(blockIdx.x);
    begin();
    int stores = 0;  // of the tile before, behind the loads of begin()
    for (uint32_t id = blockIdx.x;;) {
#pragma unroll
        for (int part = 0; part < SOON; ++part) fetch_part(std::false_type{}, part, 0, NB - 1);
        if (LOOP && stores) lds_landed_but<SOON + OM * (FN / FS) * STORES>();
        else lds_landed_but<(NB - 2) * LOADS + SOON>();
        read_scales(0, sb, sa);
        mine(sb, sa);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
#pragma unroll
        for (int j = 0; j < FM; ++j) fa[0][j] = read_a(1 % NB, wk * STEPS, j);
#pragma unroll
        for (int i = 0; i < FN; ++i) fb[0][i] = read_b(std::false_type{}, 1 % NB, wk * STEPS, i, 0);
        // fast stages: where rows of scales end inside a piece, those whose chunks are whole
        const int fast_end = min(whole, slen % 16 == 0 ? whole : slen / kScaleBytes * kChunk - kChunk);
        int s = 0;
        for (; s + 2 * NB - 1 < fast_end; s += NB) {
#pragma unroll
            for (int u = 0; u < NB; ++u) stage((u + 1) % NB, (u + 2) % NB, std::true_type{}, s + u);
        }
#pragma unroll 1
        for (; s < stages; ++s) stage((s + 1) % NB, (s + 2) % NB, std::false_type{}, s);
        lds_landed();  // every wave has read its last fragments, and no load is on its way
        const int64_t n_here = n0, m_here = m0;
        id += gridDim.x;
        const bool more = LOOP && id < tn * tm;
        if (more) {  // the next tile's first loads, on their way while this one is stored
            go_to(id);
            begin();
        }

        // Two waves with parts of one sum exchange halves of it, tokens by tokens.
        if constexpr (KW == 2) {
            static_assert(NW * FN * OM * 4096 <= NB * STAGE, "exchange");
            f32x4* out = reinterpret_cast<f32x4*>(lds + w * (FN * OM * 4096)) + l;
            const f32x4* in = reinterpret_cast<const f32x4*>(lds + (w ^ 1) * (FN * OM * 4096)) + l;
#pragma unroll
            for (int j = 0; j < OM; ++j)
#pragma unroll
                for (int i = 0; i < FN; ++i) {
                    f32x16 give;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        give[e] = wk ? acc[i][j][e] : acc[i][j + OM][e];
                        acc[i][j][e] = wk ? acc[i][j + OM][e] : acc[i][j][e];
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        out[((j * FN + i) * 4 + q) * WAVE] =
                            f32x4{give[4 * q], give[4 * q + 1], give[4 * q + 2], give[4 * q + 3]};
                }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < OM; ++j)
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = in[((j * FN + i) * 4 + q) * WAVE];
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
                    }
            __syncthreads();
        }

        // 32 tokens at a time through the wave's part of LDS, so that a store takes
        // whole 16-byte pieces of a few rows of C.  Piece p of row r in slot p ^ r.
        uint8_t* own = lds + w * (32 * RB);
        int lane = l;  // opaque, as in go_to
        asm volatile("" : "+v"(lane));
        const bool inside = n_here + BN <= g.b.rows && m_here + BM <= g.a.rows;
#pragma unroll
        for (int ji = 0; ji < OM * (FN / FS); ++ji) {
            const int j = ji / (FN / FS), i0 = ji % (FN / FS) * FS;
            const int64_t row0 = m_here + (wm * FM + wk * OM + j) * 32, col0 = n_here + (wn * FN + i0) * 32;
            // where store q of this lane goes, and how many columns there are
            auto place = [&](int q, T*& to) {
                const int r = (q * WAVE + lane) / PR, p = (q * WAVE + lane) % PR;
                const int64_t row = row0 + r, col = col0 + p * E;
                to = c + row * g.ldc + col;
                return inside || row < g.a.rows ? g.b.rows - col : (int64_t)0;
            };
#pragma unroll
            for (int i = 0; i < FS; ++i) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i0 + i][j][4 * q + e];
                    const int at = (i * 32 + q * 8 + 4 * (lane >> 5)) * (int)sizeof(T), r = lane & 31;
                    const auto four = packed4(c, v);
                    *reinterpret_cast<std::remove_const_t<decltype(four)>*>(
                        own + r * RB + (((at >> 4) ^ (r & (PR - 1))) << 4) + (at & 15)) = four;
                }
            }
            wave_lds_sync();
            auto piece = [&](int q) {
                const int r = (q * WAVE + lane) / PR, p = (q * WAVE + lane) % PR;
                return own + r * RB + ((p ^ (r & (PR - 1))) << 4);
            };
            if (ADD && inside) {
                // what is there: eight loads before the first store, which the compiler
                // could move no load ahead of (4096 x 4096 x 4096: 65 us with each load
                // before its store)
                constexpr int AT = STORES < 8 ? STORES : 8;
#pragma unroll
                for (int q = 0; q < STORES; q += AT) {
                    u32x4 old[AT];
                    T* to[AT];
#pragma unroll
                    for (int e = 0; e < AT; ++e) {
                        place(q + e, to[e]);
                        old[e] = *reinterpret_cast<const u32x4_a2*>(to[e]);
                    }
#pragma unroll
                    for (int e = 0; e < AT; ++e) {
                        u32x4 v = *reinterpret_cast<const u32x4*>(piece(q + e));
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            v[f] = __float_as_uint(__uint_as_float(old[e][f]) + __uint_as_float(v[f]));
                        *reinterpret_cast<u32x4_a2*>(to[e]) = v;
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < STORES; ++q) {
                    T* to;
                    const int64_t left = place(q, to);
                    if (!ADD && (inside || left >= E)) {
                        *reinterpret_cast<u32x4_a2*>(to) = *reinterpret_cast<const u32x4*>(piece(q));
                    } else {
                        for (int e = 0; e < E; ++e)
                            if (e < left) put_result<ADD>(to + e, to_f32(reinterpret_cast<const T*>(piece(q))[e]));
                    }
                }
            }
            wave_lds_sync();
        }
        if (!more) break;
        stores = inside;
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // buffer 0 is free
    }
}

template <class T, bool ADD, int BN, int BM, int WN, int WM, int KW, int NB>
hipError_t launch_pipe(const Args& g, int splits, T* c, hipStream_t stream) {
    int64_t tiles = ((g.b.rows + BN - 1) / BN) * ((g.a.rows + BM - 1) / BM);
    if (KW == 1 && NB == 2 && splits == 1 && tiles > kUnits) tiles = kUnits;  // the blocks go on to the others
    hipLaunchKernelGGL((k_mm_mx_pipe<T, ADD, BN, BM, WN, WM, KW, NB>), dim3((unsigned)tiles, splits),
                       dim3(WN * WM * KW * WAVE), 0, stream, g, c);
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
            if constexpr (ADD) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += to[min((int64_t)e, g.b.rows - 1 - col)];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < g.b.rows) put_result<false>(to + e, sum[e]);
        }
    }
}

template <class T, bool ADD, int NT, int MT, int WS, int NB>
hipError_t launch_few(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.b.rows + NT * 16 - 1) / (NT * 16)) * ((g.a.rows + MT * 16 - 1) / (MT * 16));
    hipLaunchKernelGGL((k_mm_mx_few<T, ADD, NT, MT, WS, NB>), dim3((unsigned)tiles), dim3(WS * WAVE), 0, stream, g, c);
    return hipGetLastError();
}

// The same for up to R tokens that are encoded on the way.  Every block encodes
// them anew, but x lies in L2 after the first one has read it, and a launch is
// saved.  For each slab a wave's lanes hold 8 values of a token each (a group
// is four lanes, as in the encoder); codes and scale bytes go through the wave's
// part of LDS, laid out as the loads of the kernel above would.  (With each
// lane encoding the groups that it multiplies, all 16 rows of a tile whether
// there are tokens or not, one token x 4096 x 4096 took 5.9 us.)
struct X {
    const void* x;
    int64_t ldx, k;
};

template <class T, class V, int NT, int R, int WS, int NB>
__global__ void __launch_bounds__(WS * WAVE)
k_mm_mx_fused(Args g, X x, T* __restrict__ c) {
    typedef SlabLoader<NT * 16> LB;
    constexpr int SLAB = LB::BYTES, TOKENS = R * (kSlab + 16);
    constexpr int ALL = NB * SLAB + TOKENS, OWN = ALL > NT * 1024 ? ALL : NT * 1024;
    static_assert(WS * OWN <= 160 * 1024 && OWN % 16 == 0 && R <= 16, "LDS");
    __shared__ __align__(1024) uint8_t lds[WS * OWN];
    const int l = lane_id(), quad = l >> 4, w = __builtin_amdgcn_readfirstlane(wave_id());
    const int64_t n0 = (int64_t)blockIdx.x * (NT * 16);
    const int pitch = (int)g.pitch, spitch = (int)g.spitch;
    LB lb;
    lb.init(g.b, n0, g.pitch, g.spitch);
    uint8_t* own = lds + w * OWN;
    uint8_t* tokens = own + NB * SLAB;

    f32x4 acc[NT] = {};
    const int slabs = (pitch + kSlab - 1) / kSlab;
    const int mine = (slabs - w + WS - 1) / WS;  // slabs w, w + WS, ...
#pragma unroll
    for (int b = 0; b < NB; ++b)
        if (b < mine) lb.load(w + b * WS, lds_addr(own) + b * SLAB, pitch, spitch);
    Raw8<V> v[R];
    auto load_values = [&](int slab) {
        const int64_t at = (int64_t)slab * (2 * kSlab) + 8 * l;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = min((int64_t)r, g.a.rows - 1);
            v[r].template load<false>(static_cast<const V*>(x.x) + row * x.ldx + at, x.k - at, at > 0);
        }
    };
    if (mine > 0) load_values(w);
    for (int it = 0; it < mine; ++it) {
        const int slab = w + it * WS, buf = it % NB;
        const int64_t first = (int64_t)slab * (2 * kSlab) + 8 * l;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r].settle(x.k - first, first > 0);
            const uint32_t byte = mx_byte(quad_max(v[r].amax_bits()));
            const uint32_t word = v[r].codes(mx_scale(byte));
            *reinterpret_cast<uint32_t*>(tokens + r * kSlab + (((l >> 2) ^ r) << 4) + (l & 3) * 4) =
                byte == kMxNaN ? 0u : word;
            if ((l & 3) == 0) tokens[R * kSlab + r * 16 + (l >> 2)] = (uint8_t)byte;
        }
        // this slab's weights were fetched before its values, which have been used
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        if (it + 1 < mine) load_values(slab + WS);
        wave_lds_sync();
        const uint8_t* at = own + buf * SLAB;
        const bool there = slab * 16 + quad * 4 < spitch;
        const int row = min(l & 15, R - 1);
        const int sa = *reinterpret_cast<const int*>(tokens + R * kSlab + row * 16 + quad * 4);
        int sb[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int word = *reinterpret_cast<const int*>(at + NT * 16 * kSlab + i * 256 + (l & 15) * 16 + quad * 4);
            sb[i] = there ? word : 0;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int piece = quad * 4 + kk;
            const i32x4 fa = *reinterpret_cast<const i32x4*>(tokens + row * kSlab + ((piece ^ row) << 4));
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                i32x4 fb = *reinterpret_cast<const i32x4*>(at + (i * 16 + (l & 15)) * kSlab + ((piece ^ (l & 15)) << 4));
                if (slab * kSlab + piece * 16 >= pitch) fb = i32x4{0, 0, 0, 0};
                acc[i] = mfma16(kk, fb, fa, acc[i], sb[i], sa);
            }
        }
        // this slab and its tokens have been read
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        if (it + NB < mine) lb.load(slab + NB * WS, lds_addr(own) + buf * SLAB, pitch, spitch);
    }

    f32x4* sums = reinterpret_cast<f32x4*>(own);
#pragma unroll
    for (int i = 0; i < NT; ++i) sums[i * WAVE + l] = acc[i];
    __syncthreads();
    for (int f = w; f < NT; f += WS) {
        f32x4 sum = {};
#pragma unroll
        for (int s = 0; s < WS; ++s) sum += *reinterpret_cast<const f32x4*>(lds + s * OWN + (f * WAVE + l) * 16);
        const int64_t row = l & 15, col = n0 + f * 16 + 4 * quad;
        if (row < g.a.rows) {
            T* to = c + row * g.ldc + col;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < g.b.rows) put(to + e, sum[e]);
        }
    }
}

template <class T, class V, int NT, int R, int WS, int NB>
hipError_t launch_fused(const Args& g, const X& x, T* c, hipStream_t stream) {
    const dim3 grid((unsigned)((g.b.rows + NT * 16 - 1) / (NT * 16)));
    hipLaunchKernelGGL((k_mm_mx_fused<T, V, NT, R, WS, NB>), grid, dim3(WS * WAVE), 0, stream, g, x, c);
    return hipGetLastError();
}

// ------------------------------------------------------------------ splits
// Sums of the splits, in order, to c (or to what c holds).  A thread takes four
// neighbouring columns; the parts' rows are whole fours.
template <class T, bool ADD>
__global__ void __launch_bounds__(256)
k_mm_mx_join(const float* __restrict__ parts, int splits, int64_t stride, int64_t m, int64_t n, T* __restrict__ c,
             int64_t ldc) {
    const int64_t fours = (n + 3) / 4, total = m * fours;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        f32x4 sum = ld_f4(parts + i * 4);
#pragma unroll 4
        for (int s = 1; s < splits; ++s) sum += ld_f4(parts + s * stride + i * 4);
        const int64_t row = i / fours, col = i % fours * 4;
        T* to = c + row * ldc + col;
        if (n - col >= 4) {
            float v[4] = {sum[0], sum[1], sum[2], sum[3]};
            typedef decltype(packed4(to, v)) V;
            typedef V V_at_any __attribute__((aligned(sizeof(T))));
            if constexpr (ADD) {
                const f32x4 old = *reinterpret_cast<const V_at_any*>(to);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = old[e] + v[e];
            }
            *reinterpret_cast<V_at_any*>(to) = packed4(to, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < n) put_result<ADD>(to + e, sum[e]);
        }
    }
}

// ------------------------------------------------------------------ choice
// Which tile, and in how many parts k: the least of
//   first + first_k * k + (rounds - 1) * (more + more_k * k) + join,
// rounds of blocks over the 256 compute units.  `first` and `first_k` (for 1,024
// values) fit the whole time of a call of 256 blocks, weights from HBM, `more`
// and `more_k` that of a further round, of all shapes at k = 256, 1024, 4096 and
// 8192 with n = 4096 and m = 16 to 32768 (us).  Against the next best, n = k =
// 4096:
//   m   16: 16 x 16 4.4 us (32 x 16 5.2)     m   64: 32 x 32 5.9 (32 x 64 7.4)
//   m  128: 32 x 64 7.5 (32 x 32 8.9)        m  256: 64 x 64 11.0 (32 x 64 11.9)
//   m  512: 64 x 128 14.1 (64 x 64 14.3)     m 1024: 128 x 128 19.3 (128 x 256 23.6)
//   m 2048: 128 x 256 27.6 (256 x 256 32.0)  m 4096: 256 x 256 42.0 (128 x 256 53.6)
struct Shape {
    int bn, bm;  // channels, tokens
    float first, first_k, more, more_k;
};
constexpr Shape kShapes[] = {
    {16, 16, 2.4f, 0.52f, 1.2f, 0.2f},   {32, 16, 2.6f, 0.63f, 1.3f, 0.33f},   {32, 32, 2.9f, 0.8f, 1.5f, 0.47f},
    {32, 64, 3.6f, 0.97f, 2.2f, 0.65f},  {64, 64, 5.0f, 1.43f, 1.5f, 1.07f},   {64, 128, 5.6f, 2.05f, 3.6f, 1.93f},
    {128, 128, 7.2f, 2.9f, 4.5f, 2.75f}, {128, 256, 7.4f, 5.0f, 4.0f, 5.1f},   {256, 256, 10.8f, 7.6f, 8.3f, 7.5f},
};
constexpr int kAll = sizeof(kShapes) / sizeof(kShapes[0]), kFirstPipe = 4;
// Parts are joined by a launch of its own (2.5 us) that reads them at 4 TB/s (130
// x 120 x 30050 in 15 parts: 11.8 us, 2.9 to 3.8 of them the join, whose bytes
// take 0.2).
// Only the pipelined tiles are split, as the others share k among their waves;
// a part has at least four stages.
constexpr int kMaxSplits = 16, kLeastStages = 4;
constexpr int64_t kMaxGrid = (int64_t(1) << 23) - 1;  // of 512 threads: a launch has fewer than 2^32

struct Choice {
    int shape, splits, stages_per_split;
};

int64_t up4(int64_t v) { return (v + 3) / 4 * 4; }

Choice choose(int64_t m, int64_t n, int64_t k) {
    const int stages = (int)(((k + 31) / 32 * 16 + kStage - 1) / kStage);
    Choice best{kAll - 1, 1, stages};
    double least = 1e300;
    for (int i = 0; i < kAll; ++i) {
        const Shape& s = kShapes[i];
        const int64_t blocks = ((n + s.bn - 1) / s.bn) * ((m + s.bm - 1) / s.bm);
        if (blocks > kMaxGrid) continue;  // the last shape has no more
        for (int splits = 1; splits <= (i >= kFirstPipe ? kMaxSplits : 1); splits *= 2) {
            const int each = (stages + splits - 1) / splits;
            if (splits > 1 && (each < kLeastStages || blocks * splits > 2 * kUnits)) break;
            const int parts = (stages + each - 1) / each;
            const double kk = splits == 1 ? (double)k : (double)each * 2 * kStage;
            const double more = (double)((blocks * parts - 1) / kUnits);
            double us = s.first + s.first_k * kk / 1024.0 + more * (s.more + s.more_k * kk / 1024.0);
            if (parts > 1) us += 2.5 + (double)m * n * 4 * 2 * parts / 4e6;
            if (us < least) {
                best = Choice{i, parts, each};
                least = us;
            }
        }
    }
    return best;
}

template <class T, bool ADD>
hipError_t launch_shape(int shape, const Args& g, int splits, T* c, hipStream_t stream) {
    switch (shape) {
        case 0: return launch_few<T, ADD, 1, 1, 8, 2>(g, c, stream);
        case 1: return launch_few<T, ADD, 2, 1, 6, 2>(g, c, stream);
        case 2: return launch_few<T, ADD, 2, 2, 8, 1>(g, c, stream);
        case 3: return launch_few<T, ADD, 2, 4, 6, 1>(g, c, stream);
        case 4: return launch_pipe<T, ADD, 64, 64, 1, 1, 2, 4>(g, splits, c, stream);
        case 5: return launch_pipe<T, ADD, 64, 128, 1, 2, 2, 4>(g, splits, c, stream);
        case 6: return launch_pipe<T, ADD, 128, 128, 2, 2, 2, 4>(g, splits, c, stream);
        case 7: return launch_pipe<T, ADD, 128, 256, 2, 4, 1, 2>(g, splits, c, stream);
        default: return launch_pipe<T, ADD, 256, 256, 2, 4, 1, 2>(g, splits, c, stream);
    }
}

template <class T, bool ADD>
hipError_t launch(const Choice& w, Args g, T* c, int64_t ldc, float* parts, hipStream_t stream) {
    if (w.splits == 1) {
        g.ldc = ldc;
        return launch_shape<T, ADD>(w.shape, g, 1, c, stream);
    }
    const int64_t m = g.a.rows, n = g.b.rows;
    g.ldc = up4(n);
    g.split_stride = m * g.ldc;
    const hipError_t e = launch_shape<float, false>(w.shape, g, w.splits, parts, stream);
    if (e != hipSuccess) return e;
    const int64_t blocks = (m * (g.ldc / 4) + 255) / 256;
    hipLaunchKernelGGL((k_mm_mx_join<T, ADD>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream,
                       parts, w.splits, g.split_stride, m, n, c, ldc);
    return hipGetLastError();
}

Args args_of(const void* a, const void* a_scales, const void* b, const void* b_scales, int64_t m, int64_t n, int64_t k,
             int stages_per_split) {
    return Args{{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales), m},
                {static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales), n},
                (k + 31) / 32 * 16,
                (k + 127) / 128 * 4,
                0,
                stages_per_split,
                0};
}

// Up to kFew tokens are encoded by the blocks that multiply them.  In us, and in
// parentheses an encoding and a product in two launches, per call of a captured
// graph and, where the host is the slower side, per call from Python:
//                     a graph                                       from Python
//   n 4096  k 4096    1 token 2.9 (4.7), 4: 4.2 (5.1), 8: 5.5 (5.2)    8: 6.6 (9.2)
//   n 8192  k 8192    5.6 (7.8)          7.9 (8.1)     8.9 (8.2)       8.9 (9.0)
//   n 4096  k 11008   4.5 (6.4)          6.6 (6.7)     9.2 (7.2)       9.2 (9.2)
//   n 11008 k 4096    4.8 (9.3)          7.0 (9.8)     11.4 (10.3)    10.5 (9.2)
// One launch is the faster one up to 4 tokens; with 5 to 8 it saves the host 2.6
// us, and the GPU takes up to a quarter longer, as every block encodes all of
// them.  16 tokens x 4096 x 4096 from Python: 8.0 (7.0).  Blocks of 32 channels
// where those of 16 are more than the compute units and each encodes eight
// tokens (8 x 8192 x 8192 8.9 us against 15.5).
constexpr int kFew = 8;
bool takes_fused(int64_t m, int64_t n) { return m <= kFew && (n + 15) / 16 <= kMaxGrid; }

template <class T, class V>
hipError_t fused(Args g, const X& x, T* c, int64_t ldc, hipStream_t stream) {
    g.ldc = ldc;
    if (g.a.rows == 1) return launch_fused<T, V, 1, 1, 8, 2>(g, x, c, stream);
    if (g.a.rows <= 4) return launch_fused<T, V, 1, 4, 8, 2>(g, x, c, stream);
    return g.b.rows > 16 * kUnits ? launch_fused<T, V, 2, 8, 8, 1>(g, x, c, stream)
                                  : launch_fused<T, V, 1, 8, 8, 2>(g, x, c, stream);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

int64_t matmul_mxfp4_workspace(int64_t m, int64_t n, int64_t k) {
    const Choice w = choose(m, n, k);
    return w.splits > 1 ? w.splits * m * up4(n) * 4 : 0;
}

hipError_t launch_matmul_mxfp4(const void* a, const void* a_scales, const void* b, const void* b_scales, int64_t m,
                               int64_t n, int64_t k, void* c, bool bf16, int64_t ldc, bool accumulate,
                               void* workspace, hipStream_t stream) {
    const Choice w = choose(m, n, k);
    const Args g = args_of(a, a_scales, b, b_scales, m, n, k, w.stages_per_split);
    float* parts = static_cast<float*>(workspace);
    if (bf16) return launch<BF16, false>(w, g, static_cast<BF16*>(c), ldc, parts, stream);
    return accumulate ? launch<float, true>(w, g, static_cast<float*>(c), ldc, parts, stream)
                      : launch<float, false>(w, g, static_cast<float*>(c), ldc, parts, stream);
}

// Codes of x, then their scales, each from a multiple of 256 bytes on; then the product's own.
int64_t linear_mxfp4_workspace(int64_t m, int64_t n, int64_t k, bool x_bf16) {
    (void)x_bf16;
    if (takes_fused(m, n)) return 0;
    return up256(m * ((k + 31) / 32 * 16)) + up256(m * ((k + 127) / 128 * 4)) + matmul_mxfp4_workspace(m, n, k);
}

hipError_t launch_linear_mxfp4(const void* x, bool x_bf16, int64_t ldx, const void* b, const void* b_scales, int64_t m,
                               int64_t n, int64_t k, void* c, bool bf16, int64_t ldc, void* workspace,
                               hipStream_t stream) {
    if (takes_fused(m, n)) {
        const Args g = args_of(nullptr, nullptr, b, b_scales, m, n, k, 0);
        const X in{x, ldx, k};
        if (bf16)
            return x_bf16 ? fused<BF16, BF16>(g, in, static_cast<BF16*>(c), ldc, stream)
                          : fused<BF16, float>(g, in, static_cast<BF16*>(c), ldc, stream);
        return x_bf16 ? fused<float, BF16>(g, in, static_cast<float*>(c), ldc, stream)
                      : fused<float, float>(g, in, static_cast<float*>(c), ldc, stream);
    }
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + up256(m * ((k + 31) / 32 * 16));
    uint8_t* rest = scales + up256(m * ((k + 127) / 128 * 4));
    const hipError_t e = launch_encode_mxfp4(x, x_bf16, m, k, ldx, codes, scales, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    return launch_matmul_mxfp4(codes, scales, b, b_scales, m, n, k, c, bf16, ldc, false, rest, stream);
}

}  // namespace qc
