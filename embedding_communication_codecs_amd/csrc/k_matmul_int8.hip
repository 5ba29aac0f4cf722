// k_matmul_int8.hip -- C[m][n] = sa[m] * sb[n] * sum_k A[m][k] B[n][k] over INT8
// codes, both matrices with k contiguous: a linear layer on tokens (A, a
// scale per token) and weights (B, a scale per output channel).
//
// The sum is exact: v_mfma_i32_16x16x64_i8 accumulates in int32, and k is
// limited so that it cannot overflow.  The weights are the matrix
// instruction's A operand and the tokens its B operand, so a lane ends up
// with four neighbouring output channels of one token.
//
// Large products are bound by the matrix cores at the clock that the power
// budget leaves them (random codes 2.3-2.8 POP/s, all zeros 3.4: 16384 x 8192
// x 8192 785 us, 4096 x 4096 x 4096 53 us, their matrix cores busy three
// quarters of the time); a few tokens by the weights' bytes and one load's
// latency (one token x 4096 x 4096 4.8 us, 16 MB at 3.5 TB/s).
#include "qc_lds.hpp"
#include "qc_launch.hpp"

#include <type_traits>

namespace qc {
namespace {

struct Args {
    const uint8_t* a;  // tokens, m rows
    const float* sa;
    int64_t lda;
    const uint8_t* b;  // weights, n rows
    const float* sb;
    int64_t ldb;
    int64_t m, n;
    int32_t k;
    int64_t ldc;
};

// C = (sum * sa) * sb: the scales are applied one after the other, so that
// two tiny ones cannot underflow together.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) { return ((float)sum * sa) * sb; }

__device__ __forceinline__ u32x2 packed4(const BF16*, const float (&v)[4]) {
    return u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}
__device__ __forceinline__ f32x4 packed4(const float*, const float (&v)[4]) { return f32x4{v[0], v[1], v[2], v[3]}; }

// Four values, `left` of which exist, in one store wherever they start.
template <class T>
__device__ __forceinline__ void store4(T* p, int left, const float (&v)[4]) {
    typedef decltype(packed4(p, v)) V;
    typedef V V_at_any __attribute__((aligned(sizeof(T))));
    if (left >= 4) {
        *reinterpret_cast<V_at_any*>(p) = packed4(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) put(p + i, v[i]);
    }
}

// Rows of a matrix lie in LDS as K bytes (128 or 256), their 16-byte pieces
// permuted so that the fragment reads are free of bank conflicts: a
// ds_read_b128 takes, in one go, a piece of eight neighbouring rows and the
// piece beside it of eight others; these 16 have to differ modulo 256 bytes.
template <int K>
__device__ __forceinline__ int slot_of(int row, int piece) {
    static_assert(K == 128 || K == 256, "row bytes");
    return piece ^ (K == 128 ? row & 7 : (2 * row) & 15);
}

// Rows [row0, row0 + ROWS) of a matrix, K bytes from k0 of each, into LDS by
// NW waves; a load takes 1,024 / K rows.  Rows past the matrix repeat its
// last row (their results are not stored) and pieces past a row's padded end
// repeat its last piece (made zeros before use), so every address is inside
// the matrix.  Buffer addressing: a lane's offset inside the tile in a VGPR,
// k0 in an SGPR.
//
// What bounds these kernels is the rate at which a compute unit loads, and
// that depends on how much of a row a load takes.  Measured from L2, 256
// rows 8 KiB apart, all compute units at work: 16 rows x 64 bytes a load 50
// bytes/ns a compute unit, 8 x 128 72, 4 x 256 134, 1 x 1,024 148.
template <int ROWS, int K, int NW>
struct Loader {
    static constexpr int RPL = 1024 / K, N = ROWS / RPL / NW;  // rows a load, loads a wave
    static_assert(N >= 1 && N * RPL * NW == ROWS, "every wave loads alike");
    int off[N];
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ void init(const uint8_t* mat, int64_t ld, int64_t row0, int64_t rows, int padded,
                                         int wave) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = min(row(wave, i), last) * (int)ld + piece(wave, i) * 16;
        rsrc = buffer_of(mat + row0 * ld, last * (int)ld + padded);
    }
    __device__ __forceinline__ static int row(int wave, int i) { return (wave * N + i) * RPL + lane_id() / (K / 16); }
    __device__ __forceinline__ static int piece(int wave, int i) {
        return slot_of<K>(row(wave, i), lane_id() % (K / 16));
    }
    // load `i` of N at k0.  WHOLE: the rows reach k0 + K.
    template <bool WHOLE>
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, int k0, int padded) const {
        const int over = WHOLE ? 0 : max(k0 + piece(wave, i) * 16 - (padded - 16), 0);
        load_lds16(rsrc, lds + (wave * N + i) * 1024, off[i] - over, k0);
    }
};

// Of four neighbouring codes, those at k and after become zeros; `at`: where the first is.
__device__ __forceinline__ uint32_t cut_word(uint32_t word, int at, int k) {
    const int keep = k - at;
    return keep <= 0 ? 0u : (keep >= 4 ? word : word & ((1u << (8 * keep)) - 1u));
}

// The same for a tile of ROWS rows in LDS, `valid` of K bytes of which exist.
template <int ROWS, int K, int THREADS>
__device__ __forceinline__ void zero_tail(uint8_t* lds, int valid) {
    for (int i = threadIdx.x; i < ROWS * (K / 16); i += THREADS) {
        const int r = i / (K / 16), c = i % (K / 16);
        u32x4* p = reinterpret_cast<u32x4*>(lds + r * K + (slot_of<K>(r, c) << 4));
        if (c * 16 + 16 > valid) {
            u32x4 v = *p;
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] = cut_word(v[w], c * 16 + w * 4, valid);
            *p = v;
        }
    }
}

// ------------------------------------------------------- pipelined tiles
// One block computes BN channels x BM tokens with WN x WM waves, in stages of
// K bytes of k, NB of them in LDS.  A wave reads its fragments ahead of their
// use, into the next stage too; the wait for that stage, and the only
// barrier, stand where the last fragments of this one have been read, and the
// fragments already in registers keep the matrix cores busy across it.  The
// loads of the stage NB further on follow at once, over the one just left,
// and have NB - 1 stages' time to arrive: a stage of a small tile is shorter
// than a load takes, so it needs more of them (1024 x 4096 x 4096 with tiles
// of 128 x 128: 21.6 us with four stages of 128 bytes, 25 with two of 256;
// 256 x 4096 x 4096 with 64 x 64: 12.5 with four, 15.8 with two of 256).
template <class T, int BN, int BM, int WN, int WM, int K, int NB>
__global__ void __launch_bounds__(WN * WM * WAVE)
k_mm_int8_pipe(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FM = BM / WM / 16;
    constexpr int AHEAD = FN >= 8 ? 3 : 2;                 // weight fragments read ahead (of a ring of 4)
    constexpr int KK = K / 64, STEPS = KK * FN;            // a step: one weight fragment
    constexpr int TURN = STEPS - FN / 2;                   // the barrier's step
    constexpr int TB = BN * K, STAGE = (BN + BM) * K;      // weights first, then tokens
    // a stage's last read comes before the barrier, the next one's first after it
    static_assert(FN % 4 == 0 && FM >= 1 && STEPS - 1 - AHEAD <= TURN && STEPS - AHEAD >= TURN, "tile shape");
    __shared__ __align__(1024) uint8_t lds[NB * STAGE];

    const uint32_t tn = (uint32_t)((g.n + BN - 1) / BN), tm = (uint32_t)((g.m + BM - 1) / BM);
    const Tile2 tile = tile_of<4>(blockIdx.x, tn, tm);
    const int64_t n0 = (int64_t)tile.x * BN, m0 = (int64_t)tile.y * BM;
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wm = w / WN;
    const int l = lane_id();
    const int padded = (g.k + 15) & ~15;
    Loader<BN, K, NW> lb;
    Loader<BM, K, NW> la;
    constexpr int LOADS = lb.N + la.N;
    lb.init(g.b, g.ldb, n0, g.n, padded, w);
    la.init(g.a, g.lda, m0, g.m, padded, w);

    const int stages = (g.k + K - 1) / K;
    const int whole = g.k / K;  // a stage from here on (one at most) holds bytes past k
    const uint32_t lds0 = lds_addr(lds);
    auto fetch_part = [&](auto fast, int part, int buf, int s) {  // one of LOADS
        constexpr bool FAST = decltype(fast)::value;
        if (part < lb.N) lb.template load<FAST>(part, lds0 + buf * STAGE, w, s * K, padded);
        else la.template load<FAST>(part - lb.N, lds0 + buf * STAGE + TB, w, s * K, padded);
    };
    auto fetch = [&](int s) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) fetch_part(std::false_type{}, part, s % NB, s);
    };
    auto cut = [&](int s) {
        if (s >= whole) {  // the weights' bytes past k become zeros (integers: one side is enough)
            zero_tail<BN, K, THREADS>(lds + s % NB * STAGE, g.k - s * K);
            __syncthreads();
        }
    };

    // fragments: row l % 16, piece kk * 4 + l / 16 (an xor of kk * 64 in the address)
    const int frag = (l & 15) * K + (slot_of<K>(l & 15, l >> 4) << 4);
    const int rb = wn * FN * 16 * K + frag, ra = TB + wm * FM * 16 * K + frag;
    auto read_b = [&](int buf, int q) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (rb ^ (q / FN * 64)) + q % FN * (16 * K));
    };
    auto read_a = [&](int buf, int kk, int j) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (ra ^ (kk * 64)) + j * (16 * K));
    };

    i32x4 acc[FN][FM] = {};
    i32x4 fb[4], fa[2][FM];
    // Stage s in buffer `buf`, the next one in `next`.  FAST: stages up to s +
    // NB exist and are whole.
    auto stage = [&](int buf, int next, auto fast, int s) {
        constexpr bool FAST = decltype(fast)::value;
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int kk = q / FN, i = q % FN;
            if (q + AHEAD < STEPS) fb[(q + AHEAD) % 4] = read_b(buf, q + AHEAD);
            if (q == TURN && (FAST || s + 1 < stages)) {
                if (FAST || s + NB - 1 < stages) lds_landed_but<(NB - 2) * LOADS>();
                else lds_landed();
                if (!FAST) cut(s + 1);
            }
            if (q + AHEAD >= STEPS) fb[(q + AHEAD) % 4] = read_b(next, q + AHEAD - STEPS);
            if (i >= FN / 2) {
                constexpr int H = FN / 2;  // this step's share of the token fragments and of the loads
#pragma unroll
                for (int e = (i - H) * FM / H; e < (i - H + 1) * FM / H; ++e)
                    fa[(kk + 1) & 1][e] = kk + 1 < KK ? read_a(buf, kk + 1, e) : read_a(next, 0, e);
                if (kk + 1 == KK && (FAST || s + NB < stages)) {
#pragma unroll
                    for (int d = (i - H) * LOADS / H; d < (i - H + 1) * LOADS / H; ++d)
                        fetch_part(fast, d, buf, s + NB);
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[q % 4], fa[kk & 1][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
        }
    };

    for (int s = 0; s < NB && s < stages; ++s) fetch(s);
    if (stages >= NB) lds_landed_but<(NB - 1) * LOADS>();
    else lds_landed();
    cut(0);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[0][j] = read_a(0, 0, j);
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) fb[q] = read_b(0, q);
    int s = 0;
    for (; s + 2 * NB - 1 < whole; s += NB) {
#pragma unroll
        for (int u = 0; u < NB; ++u) stage(u, (u + 1) % NB, std::true_type{}, s + u);
    }
#pragma unroll 1
    for (; s < stages; ++s) stage(s % NB, (s + 1) % NB, std::false_type{}, s);

    // every scale before the first store: a load after a store would wait for it
    float sa[FM];
    f32x4 sb[FN];
#pragma unroll
    for (int j = 0; j < FM; ++j) sa[j] = g.sa[min(m0 + (wm * FM + j) * 16 + (l & 15), g.m - 1)];
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        const int64_t col = n0 + (wn * FN + i) * 16 + 4 * (l >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) sb[i][e] = g.sb[min(col + e, g.n - 1)];
    }
    // 16 tokens at a time through the wave's part of LDS, so that a store takes
    // whole 16-byte pieces of a few rows of C, wherever they start, and not
    // eight bytes of 16 rows (4096 x 4096 x 128: 11.5 us against 15.0; 16384 x
    // 8192 x 8192 827 against 851; 1280 x 3206 x 3776 30.5 against 38.7).  Piece
    // p of row r in slot p ^ r.
    constexpr int COLS = FN * 16, RB = COLS * (int)sizeof(T), PR = RB / 16, E = 16 / (int)sizeof(T);
    static_assert((PR & (PR - 1)) == 0 && PR <= WAVE && NW * 16 * RB <= NB * STAGE, "a wave's part of LDS");
    __syncthreads();  // every wave has read its last fragments
    uint8_t* own = lds + w * (16 * RB);
    const bool inside = n0 + BN <= g.n && m0 + BM <= g.m;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sa[j], sb[i][e]);
            const int at = (i * 16 + 4 * (l >> 4)) * (int)sizeof(T), r = l & 15;
            const auto four = packed4(c, v);
            *reinterpret_cast<std::remove_const_t<decltype(four)>*>(own + r * RB + (((at >> 4) ^ (r & (PR - 1))) << 4) +
                                                                    (at & 15)) = four;
        }
        wave_lds_sync();
        const int64_t row0 = m0 + (wm * FM + j) * 16, col0 = n0 + wn * COLS;
#pragma unroll
        for (int q = 0; q < RB / 64; ++q) {
            const int r = (q * WAVE + l) / PR, p = (q * WAVE + l) % PR;
            const uint8_t* from = own + r * RB + ((p ^ (r & (PR - 1))) << 4);
            const int64_t row = row0 + r, col = col0 + p * E, left = inside || row < g.m ? g.n - col : 0;
            T* to = c + row * g.ldc + col;
            if (inside || left >= E) {
                *reinterpret_cast<u32x4_a2*>(to) = *reinterpret_cast<const u32x4*>(from);
            } else {
                for (int e = 0; e < E; ++e)
                    if (e < left) to[e] = reinterpret_cast<const T*>(from)[e];
            }
        }
        wave_lds_sync();
    }
}

template <class T, int BN, int BM, int WN, int WM, int K, int NB>
hipError_t launch_pipe(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
    hipLaunchKernelGGL((k_mm_int8_pipe<T, BN, BM, WN, WM, K, NB>), dim3((unsigned)tiles), dim3(WN * WM * WAVE), 0,
                       stream, g, c);
    return hipGetLastError();
}

// ------------------------------------------------------------- few tokens
// One block: NT * 16 channels x MT * 16 tokens, k split over WS waves in
// slabs of 256 bytes, joined through LDS.  A wave loads the rows of its slab
// into a part of LDS of its own (no barrier until the waves join), up to NB
// slabs at a time, as 4 rows x 256 bytes a load; that pattern is what makes
// this fast: with the fragments loaded straight into registers, 16 rows x 64
// bytes a load, 61 tokens x 4096 x 4096 took 13.5 us instead of 8.5.
template <class T, int NT, int MT, int WS, int NB>
__global__ void __launch_bounds__(WS * WAVE)
k_mm_int8_few(Args g, T* __restrict__ c) {
    constexpr int K = 256, ROWS = (NT + MT) * 16, SLAB = ROWS * K;
    constexpr int OWN = NB * SLAB > NT * MT * 1024 ? NB * SLAB : NT * MT * 1024;  // a wave's LDS: slabs, then sums
    __shared__ __align__(1024) uint8_t lds[WS * OWN];
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const uint32_t tn = (uint32_t)((g.n + NT * 16 - 1) / (NT * 16));
    const int64_t n0 = (int64_t)(blockIdx.x % tn) * (NT * 16), m0 = (int64_t)(blockIdx.x / tn) * (MT * 16);
    const int padded = (g.k + 15) & ~15;
    Loader<NT * 16, K, 1> lb;
    Loader<MT * 16, K, 1> la;
    constexpr int LOADS = lb.N + la.N;
    lb.init(g.b, g.ldb, n0, g.n, padded, 0);
    la.init(g.a, g.lda, m0, g.m, padded, 0);
    uint8_t* own = lds + w * OWN;
    auto fetch = [&](int slab, int buf) {
        const uint32_t at = lds_addr(own) + buf * SLAB;
#pragma unroll
        for (int i = 0; i < lb.N; ++i) lb.template load<false>(i, at, 0, slab * K, padded);
#pragma unroll
        for (int i = 0; i < la.N; ++i) la.template load<false>(i, at + NT * 16 * K, 0, slab * K, padded);
    };

    i32x4 acc[NT][MT] = {};
    const int slabs = (g.k + K - 1) / K;
    const int mine = (slabs - w + WS - 1) / WS;  // slabs w, w + WS, ...
#pragma unroll
    for (int b = 0; b < NB; ++b)
        if (b < mine) fetch(w + b * WS, b);
    for (int it = 0; it < mine; ++it) {
        const int slab = w + it * WS, buf = NB == 1 ? 0 : it % NB;
        if (NB > 1 && it + NB <= mine) asm volatile("s_waitcnt vmcnt(%0)" : : "n"((NB - 1) * LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        const uint8_t* at = own + buf * SLAB + (l & 15) * K;
#pragma unroll
        for (int kk = 0; kk < K / 64; ++kk) {
            const int slot = slot_of<K>(l & 15, kk * 4 + (l >> 4)) << 4;
            i32x4 fb[NT], fa[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) fb[i] = *reinterpret_cast<const i32x4*>(at + i * (16 * K) + slot);
#pragma unroll
            for (int j = 0; j < MT; ++j) fa[j] = *reinterpret_cast<const i32x4*>(at + (NT + j) * (16 * K) + slot);
            if ((slab + 1) * K > g.k) {  // the weights' bytes past k become zeros
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        fb[i][e] = (int)cut_word(fb[i][e], slab * K + kk * 64 + (l >> 4) * 16 + e * 4, g.k);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i], fa[j], acc[i][j], 0, 0, 0);
        }
        if (it + NB < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // this slab has been read
            fetch(slab + NB * WS, buf);
        }
    }

    // all of a wave's loads have landed and been read; its part of LDS takes its sums
    i32x4* sums = reinterpret_cast<i32x4*>(own);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) sums[(i * MT + j) * WAVE + l] = acc[i][j];
    __syncthreads();
    for (int f = w; f < NT * MT; f += WS) {
        i32x4 sum = {};
#pragma unroll
        for (int s = 0; s < WS; ++s) sum += *reinterpret_cast<const i32x4*>(lds + s * OWN + (f * WAVE + l) * 16);
        const int64_t row = m0 + (f % MT) * 16 + (l & 15);
        const int64_t col = n0 + (f / MT) * 16 + 4 * (l >> 4);
        const int64_t left = g.n - col;
        if (row < g.m && left > 0) {
            const float sa = g.sa[row];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(sum[e], sa, e < left ? g.sb[col + e] : 0.0f);
            store4(c + row * g.ldc + col, left < 4 ? (int)left : 4, v);
        }
    }
}

template <class T, int NT, int MT, int WS, int NB>
hipError_t launch_few(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.n + NT * 16 - 1) / (NT * 16)) * ((g.m + MT * 16 - 1) / (MT * 16));
    hipLaunchKernelGGL((k_mm_int8_few<T, NT, MT, WS, NB>), dim3((unsigned)tiles), dim3(WS * WAVE), 0, stream, g, c);
    return hipGetLastError();
}

// Which tile: the one whose rounds of blocks over the 256 compute units take
// the least time.  `round_us` is the measured time of one full round at k =
// 4096 without the launch itself (2 us).  A round has a part that does not
// depend on k, and the few-token shapes share k among their waves in slabs of
// 256 bytes, but the shapes keep their order: of all nine at k = 32, 64, 128, 256,
// 512, 1024 and 4096, for 1 to 16384 tokens and n of 4096 and 8192, the one taken
// was within 5% of the best, but at 61 x 8192 x 128 (4.2 us, 64 x 64 3.8).  16384
// x 4096 x 128, for one: 256 x 256 34.4 us, 128 x 256 41.8, 128 x 128 56.4.
// Against the next best shape, whole calls, weights from HBM, at n = k = 4096
// (16384 where it says so):
//   m    1: 16 x 16 5.6 us (32 x 16 6.2)     m  16 (16384): 32 x 16 13.5 (32 x 32 15.5)
//   m   32: 32 x 16 6.7 (32 x 32 8.4)        m  32 (16384): 32 x 32 16.4 (32 x 64 17.1)
//   m   61: 32 x 32 8.4 (32 x 64 9.7)        m 128: 32 x 64 9.6 (64 x 64 12.4)
//   m  256: 64 x 64 12.5 (32 x 64 16.0)      m 512: 64 x 128 16.0 (64 x 64 19.5)
//   m 1024: 128 x 128 21.6 (128 x 256 29.1)  m 2048: 128 x 256 34.3 (128 x 128 44.2)
//   m 4096: 256 x 256 55.9 (128 x 256 67.2)
struct Shape {
    int bn, bm;  // channels, tokens
    float round_us;
};
constexpr int kUnits = 256;  // compute units, each with one block at work
constexpr Shape kShapes[] = {
    {16, 16, 4.0f},   {32, 16, 4.7f},    {32, 32, 6.5f},    {32, 64, 7.4f},    {64, 64, 10.4f},
    {64, 128, 14.1f}, {128, 128, 19.7f}, {128, 256, 32.2f}, {256, 256, 51.0f},
};

int shape_of(int64_t m, int64_t n) {
    constexpr int kAll = sizeof(kShapes) / sizeof(kShapes[0]);
    int best = kAll - 1;
    double least = 1e300;
    for (int i = 0; i < kAll; ++i) {
        const Shape& s = kShapes[i];
        const int64_t blocks = ((n + s.bn - 1) / s.bn) * ((m + s.bm - 1) / s.bm);
        const double us = (double)((blocks + kUnits - 1) / kUnits) * s.round_us;
        if (us < least && blocks < int64_t(1) << 23) {  // a grid has fewer than 2^32 threads; the last shape has
            best = i;
            least = us;
        }
    }
    return best;
}

template <class T>
hipError_t launch(const Args& g, T* c, hipStream_t stream) {
    switch (shape_of(g.m, g.n)) {
        case 0: return launch_few<T, 1, 1, 8, 2>(g, c, stream);
        case 1: return launch_few<T, 2, 1, 6, 2>(g, c, stream);
        case 2: return launch_few<T, 2, 2, 8, 1>(g, c, stream);
        case 3: return launch_few<T, 2, 4, 6, 1>(g, c, stream);
        case 4: return launch_pipe<T, 64, 64, 1, 4, 128, 4>(g, c, stream);
        case 5: return launch_pipe<T, 64, 128, 1, 4, 128, 4>(g, c, stream);
        case 6: return launch_pipe<T, 128, 128, 2, 4, 128, 4>(g, c, stream);
        case 7: return launch_pipe<T, 128, 256, 2, 4, 128, 3>(g, c, stream);
        default: return launch_pipe<T, 256, 256, 2, 4, 128, 2>(g, c, stream);
    }
}

}  // namespace

hipError_t launch_matmul_int8(const void* a, const float* a_scale, int64_t lda, const void* b, const float* b_scale,
                              int64_t ldb, int64_t m, int64_t n, int64_t k, void* c, bool bf16, int64_t ldc,
                              hipStream_t stream) {
    const Args g{static_cast<const uint8_t*>(a), a_scale, lda, static_cast<const uint8_t*>(b), b_scale, ldb, m, n,
                 (int32_t)k, ldc};
    return bf16 ? launch(g, static_cast<BF16*>(c), stream) : launch(g, static_cast<float*>(c), stream);
}

}  // namespace qc
