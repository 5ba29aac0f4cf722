// k_matmul_int8.hip -- C[m][n] = sa[m] * sb[n] * sum_k A[m][k] B[n][k] over INT8
// codes, both matrices with k contiguous: a linear layer on tokens (A, a
// scale per token) and weights (B, a scale per output channel).
//
// The sum is exact: v_mfma_i32_16x16x64_i8 accumulates in int32, and k is
// limited so that it cannot overflow.  The weights are the matrix
// instruction's A operand and the tokens its B operand, so a lane ends up
// with four neighbouring output channels of one token.
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
    bool wide;  // rows of C start at multiples of four elements
};

// C = (sum * sa) * sb: the scales are applied one after the other, so that
// two tiny ones cannot underflow together.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) { return ((float)sum * sa) * sb; }

__device__ __forceinline__ void store4(BF16* p, int left, const float (&v)[4], bool wide) {
    if (wide && left >= 4) {
        *reinterpret_cast<u32x2*>(p) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) put(p + i, v[i]);
    }
}
__device__ __forceinline__ void store4(float* p, int left, const float (&v)[4], bool wide) {
    if (wide && left >= 4) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = v[i];
    }
}

constexpr int BK = 128;  // bytes of k per step: one LDS row, eight 16-byte pieces

// Rows [row0, row0 + ROWS) of a matrix, bytes [k0, k0 + 128) of each, into
// LDS.  A wave's load writes 1,024 consecutive LDS bytes, eight rows; piece
// c of row r goes to slot c ^ (r & 7), so that the fragment reads (16 rows,
// one piece each) spread over all banks.  Rows past the matrix repeat its
// last row (their results are not stored) and pieces past the row's padded
// end repeat its last piece (zeroed in LDS before use), so every address is
// inside the matrix.  Buffer addressing: a lane's offset inside the tile in a
// VGPR, k0 in an SGPR.
template <int ROWS, int NW>
struct Loader {
    static constexpr int N = ROWS / 8 / NW;  // loads per wave
    int off[N];
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ void init(const uint8_t* mat, int64_t ld, int64_t row0, int64_t rows, int padded,
                                         int wave) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
        const int lrow = lane_id() >> 3, piece = (lane_id() & 7) ^ lrow;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = min((wave * N + i) * 8 + lrow, last) * (int)ld + piece * 16;
        rsrc = buffer_of(mat + row0 * ld, last * (int)ld + padded);
    }
    // load `i` of N; `over`: how far this lane's piece at k0 lies past the last one of the row
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, int k0, int over) const {
        load_lds16(rsrc, lds + (wave * N + i) * 1024, off[i] - over, k0);
    }
};

// Zeroes the bytes from `valid` (of 128) on in every row of an LDS tile.
template <int ROWS, int THREADS>
__device__ __forceinline__ void zero_tail(uint8_t* lds, int valid) {
    for (int i = threadIdx.x; i < ROWS * 8; i += THREADS) {
        const int r = i >> 3, c = i & 7;
        uint32_t* p = reinterpret_cast<uint32_t*>(lds + r * 128 + ((c ^ (r & 7)) << 4));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int keep = valid - (c * 16 + w * 4);  // bytes of this word that stay
            if (keep <= 0) p[w] = 0u;
            else if (keep < 4) p[w] &= (1u << (8 * keep)) - 1u;
        }
    }
}

// One block computes BN channels x BM tokens with WN x WM waves.
template <class T, int BN, int BM, int WN, int WM>
__global__ void __launch_bounds__(WN * WM * WAVE)
k_mm_int8(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FM = BM / WM / 16;
    constexpr int TB = BN * BK, TILE = (BN + BM) * BK;  // weights first, then tokens
    __shared__ __align__(1024) uint8_t lds[2 * TILE];
    const int64_t tn = (g.n + BN - 1) / BN;
    const int64_t tile = blockIdx.x;
    const int64_t n0 = (tile % tn) * BN, m0 = (tile / tn) * BM;
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wm = w / WN;
    const int l = lane_id();

    const int padded = (g.k + 15) & ~15;
    Loader<BN, NW> lb;
    Loader<BM, NW> la;
    lb.init(g.b, g.ldb, n0, g.n, padded, w);
    la.init(g.a, g.lda, m0, g.m, padded, w);
    const int piece16 = ((l & 7) ^ (l >> 3)) * 16;

    i32x4 acc[FN][FM] = {};
    // fragment addresses: row l%16, piece kk*4 + l/16
    const int slot = ((l >> 4) ^ (l & 7)) << 4;
    const int rb = (wn * FN * 16 + (l & 15)) * 128 + slot;
    const int ra = (wm * FM * 16 + (l & 15)) * 128 + slot;

    auto step = [&](const uint8_t* tb, const uint8_t* ta) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 fb[FN], fa[FM];
#pragma unroll
            for (int i = 0; i < FN; ++i) fb[i] = *reinterpret_cast<const i32x4*>(tb + (rb ^ (kk * 64)) + i * 2048);
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[j] = *reinterpret_cast<const i32x4*>(ta + (ra ^ (kk * 64)) + j * 2048);
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i], fa[j], acc[i][j], 0, 0, 0);
        }
    };

    const int steps = (g.k + BK - 1) / BK;
    const int tail = g.k - (steps - 1) * BK;
    const uint32_t lds0 = lds_addr(lds);
    auto fetch = [&](int buf, int t) {
        const int over = max(t * BK + piece16 - (padded - 16), 0);
#pragma unroll
        for (int i = 0; i < lb.N; ++i) lb.load(i, lds0 + buf * TILE, w, t * BK, over);
#pragma unroll
        for (int i = 0; i < la.N; ++i) la.load(i, lds0 + buf * TILE + TB, w, t * BK, over);
    };
    fetch(0, 0);
    for (int t = 0; t < steps; ++t) {
        const int buf = t & 1;
        lds_landed();
        if (t + 1 < steps) fetch(buf ^ 1, t + 1);
        if (t == steps - 1 && tail < BK) {
            // the weights' bytes past k become zeros (integers: one side is enough)
            zero_tail<BN, THREADS>(lds + buf * TILE, tail);
            __syncthreads();
        }
        step(lds + buf * TILE, lds + buf * TILE + TB);
    }

#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t row = m0 + (wm * FM + j) * 16 + (l & 15);
        if (row < g.m) {
            const float sa = g.sa[row];
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int64_t col = n0 + (wn * FN + i) * 16 + 4 * (l >> 4);
                const int64_t left = g.n - col;
                if (left > 0) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sa, e < left ? g.sb[col + e] : 0.0f);
                    store4(c + row * g.ldc + col, left < 4 ? (int)left : 4, v, g.wide);
                }
            }
        }
    }
}

template <class T, int BN, int BM, int WN, int WM>
hipError_t launch_tile(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
    hipLaunchKernelGGL((k_mm_int8<T, BN, BM, WN, WM>), dim3((unsigned)tiles), dim3(WN * WM * WAVE), 0, stream, g, c);
    return hipGetLastError();
}

// ------------------------------------------------------- pipelined tiles
// One block computes BN channels x BM tokens with WN x WM waves, in stages of
// 128 bytes of k, two of them in LDS.  A wave reads its fragments ahead of
// their use, into the next stage too; the wait for that stage, and the only
// barrier, stand where the last fragments of this one have been read, and the
// fragments already in registers keep the matrix cores busy across it.  The
// loads of the stage after next follow at once, over the one just left, and
// have a whole stage's time to arrive.
//
// 128 bytes of k and not 64: what bounds these kernels is the rate at which a
// compute unit loads, and that depends on how much of a row a load takes.
// Measured, from L2, 256 rows 8 KiB apart, all compute units: 16 rows x 64
// bytes a load 50 bytes/ns a compute unit, 8 x 128 72, 4 x 256 134.
template <class T, int BN, int BM, int WN, int WM>
__global__ void __launch_bounds__(WN * WM * WAVE)
k_mm_int8_pipe(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FM = BM / WM / 16;
    constexpr int AHEAD = FN >= 8 ? 3 : 2;                 // weight fragments read ahead (of a ring of 4)
    constexpr int STEPS = 2 * FN, TURN = STEPS - FN / 2;   // a step: one weight fragment; the barrier's step
    constexpr int TB = BN * BK, STAGE = (BN + BM) * BK;    // weights first, then tokens
    constexpr int LB = BN / 8 / NW, LOADS = (BN + BM) / 8 / NW;
    static_assert(FN % 4 == 0 && FM >= 1 && (BN / 8) % NW == 0 && (BM / 8) % NW == 0, "tile shape");
    static_assert(STEPS - 1 - AHEAD <= TURN && STEPS - AHEAD >= TURN, "a stage's last read comes before the barrier, the next one's first after it");
    __shared__ __align__(1024) uint8_t lds[2 * STAGE];

    const uint32_t tn = (uint32_t)((g.n + BN - 1) / BN), tm = (uint32_t)((g.m + BM - 1) / BM);
    const Tile2 tile = tile_of<4>(blockIdx.x, tn, tm);
    const int64_t n0 = (int64_t)tile.x * BN, m0 = (int64_t)tile.y * BM;
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wm = w / WN;
    const int l = lane_id();
    const int padded = (g.k + 15) & ~15;
    Loader<BN, NW> lb;
    Loader<BM, NW> la;
    lb.init(g.b, g.ldb, n0, g.n, padded, w);
    la.init(g.a, g.lda, m0, g.m, padded, w);
    const int piece16 = ((l & 7) ^ (l >> 3)) * 16;

    const int stages = (g.k + BK - 1) / BK;
    const int whole = g.k / BK;  // a stage from here on (one at most) holds bytes past k
    const uint32_t lds0 = lds_addr(lds);
    auto over_of = [&](int s) { return max(s * BK + piece16 - (padded - 16), 0); };
    auto fetch_part = [&](int part, int buf, int s, int over) {  // one of LOADS
        if (part < LB) lb.load(part, lds0 + buf * STAGE, w, s * BK, over);
        else la.load(part - LB, lds0 + buf * STAGE + TB, w, s * BK, over);
    };
    auto fetch = [&](int s) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) fetch_part(part, s & 1, s, over_of(s));
    };
    auto cut = [&](int s) {
        if (s >= whole) {  // the weights' bytes past k become zeros (integers: one side is enough)
            zero_tail<BN, THREADS>(lds + (s & 1) * STAGE, g.k - s * BK);
            __syncthreads();
        }
    };

    // fragment addresses: row l % 16, piece kk * 4 + l / 16
    const int frag = (l & 15) * BK + (((l >> 4) ^ (l & 7)) << 4);
    const int rb = wn * FN * 2048 + frag, ra = TB + wm * FM * 2048 + frag;
    auto read_b = [&](int buf, int q) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (rb ^ (q / FN * 64)) + q % FN * 2048);
    };
    auto read_a = [&](int buf, int kk, int j) {
        return *reinterpret_cast<const i32x4*>(lds + buf * STAGE + (ra ^ (kk * 64)) + j * 2048);
    };

    i32x4 acc[FN][FM] = {};
    i32x4 fb[4], fa[2][FM];
    // Stage s in buffer `buf`.  FAST: stages s + 1 and s + 2 exist and are whole.
    auto stage = [&](int buf, auto fast, int s) {
        constexpr bool FAST = decltype(fast)::value;
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int kk = q / FN, i = q % FN;
            if (q + AHEAD < STEPS) fb[(q + AHEAD) % 4] = read_b(buf, q + AHEAD);
            if (q == TURN && (FAST || s + 1 < stages)) {
                lds_landed();
                if (!FAST) cut(s + 1);
            }
            if (q + AHEAD >= STEPS) fb[(q + AHEAD) % 4] = read_b(buf ^ 1, q + AHEAD - STEPS);
            if (i >= FN / 2) {
                constexpr int H = FN / 2;  // this step's share of the token fragments and of the loads
#pragma unroll
                for (int e = (i - H) * FM / H; e < (i - H + 1) * FM / H; ++e)
                    fa[kk ^ 1][e] = kk == 0 ? read_a(buf, 1, e) : read_a(buf ^ 1, 0, e);
                if (kk == 1 && (FAST || s + 2 < stages)) {
#pragma unroll
                    for (int d = (i - H) * LOADS / H; d < (i - H + 1) * LOADS / H; ++d)
                        fetch_part(d, buf, s + 2, FAST ? 0 : over_of(s + 2));
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[q % 4], fa[kk][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
        }
    };

    fetch(0);
    if (stages > 1) {
        fetch(1);
        lds_landed_but<LOADS>();
    } else {
        lds_landed();
    }
    cut(0);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[0][j] = read_a(0, 0, j);
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) fb[q] = read_b(0, q);
    int s = 0;
    for (; s + 3 < whole; s += 2) {
        stage(0, std::true_type{}, s);
        stage(1, std::true_type{}, s + 1);
    }
#pragma unroll 1
    for (; s < stages; ++s) stage(s & 1, std::false_type{}, s);

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
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t row = m0 + (wm * FM + j) * 16 + (l & 15);
        T* cr = c + row * g.ldc;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int64_t col = n0 + (wn * FN + i) * 16 + 4 * (l >> 4);
            const int64_t left = row < g.m ? g.n - col : 0;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sa[j], sb[i][e]);
            store4(cr + col, left < 4 ? (int)left : 4, v, g.wide);
        }
    }
}

template <class T, int BN, int BM, int WN, int WM>
hipError_t launch_pipe(const Args& g, T* c, hipStream_t stream) {
    const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
    hipLaunchKernelGGL((k_mm_int8_pipe<T, BN, BM, WN, WM>), dim3((unsigned)tiles), dim3(WN * WM * WAVE), 0, stream, g,
                       c);
    return hipGetLastError();
}

// ------------------------------------------------------------- few tokens
// One block: NT * 16 channels x MT * 16 tokens, k split over WS waves in
// chunks of 128 bytes, joined through LDS.  Bound by the weights' bytes: they
// go from memory to the matrix instruction without LDS, two chunks of every
// row in flight a wave; the tokens come from L2.  The four lanes that hold
// a row take 32 bytes of the chunk each, half of it per instruction: the
// order of k inside a chunk is the same for both operands, and any will do.
template <class T, int NT, int MT, int WS>
__global__ void __launch_bounds__(WS * WAVE)
k_mm_int8_few(Args g, T* __restrict__ c) {
    __shared__ i32x4 part[WS * NT * MT * WAVE];
    const int l = lane_id(), w = wave_id();
    const int64_t n0 = (int64_t)blockIdx.x * (NT * 16), m0 = (int64_t)blockIdx.y * (MT * 16);
    const int padded = (g.k + 15) & ~15;
    const int chunks = (g.k + BK - 1) / BK;
    const uint8_t* pb[NT];
    const uint8_t* pa[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t r = n0 + i * 16 + (l & 15);
        pb[i] = g.b + (r < g.n ? r : g.n - 1) * g.ldb;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int64_t r = m0 + j * 16 + (l & 15);
        pa[j] = g.a + (r < g.m ? r : g.m - 1) * g.lda;
    }
    i32x4 acc[NT][MT] = {};
    struct Chunk {
        i32x4 b[NT][2], a[MT][2];
    };
    auto get = [&](Chunk& f, int ch) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = ch * BK + h * 64 + (l >> 4) * 16;
            const int in = min(at, padded - 16);  // pieces past the row repeat its last one
#pragma unroll
            for (int i = 0; i < NT; ++i) f.b[i][h] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb[i] + in));
#pragma unroll
            for (int j = 0; j < MT; ++j) f.a[j][h] = *reinterpret_cast<const i32x4*>(pa[j] + in);
        }
    };
    auto use = [&](Chunk& f, int ch) {
        if ((ch + 1) * BK > g.k) {  // the weights' bytes past k become zeros
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int keep = g.k - (ch * BK + h * 64 + (l >> 4) * 16 + e * 4);
                    const uint32_t mask = keep <= 0 ? 0u : (keep >= 4 ? ~0u : (1u << (8 * keep)) - 1u);
#pragma unroll
                    for (int i = 0; i < NT; ++i) f.b[i][h][e] &= (int)mask;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[i][h], f.a[j][h], acc[i][j], 0, 0, 0);
    };
    int ch = w;
    for (; ch + WS < chunks; ch += 2 * WS) {
        Chunk f0, f1;
        get(f0, ch);
        get(f1, ch + WS);
        use(f0, ch);
        use(f1, ch + WS);
    }
    if (ch < chunks) {
        Chunk f;
        get(f, ch);
        use(f, ch);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) part[(w * NT * MT + i * MT + j) * WAVE + l] = acc[i][j];
    __syncthreads();
    for (int f = w; f < NT * MT; f += WS) {
        i32x4 sum = part[f * WAVE + l];
#pragma unroll
        for (int s = 1; s < WS; ++s) sum += part[(s * NT * MT + f) * WAVE + l];
        const int64_t row = m0 + (f % MT) * 16 + (l & 15);
        const int64_t col = n0 + (f / MT) * 16 + 4 * (l >> 4);
        const int64_t left = g.n - col;
        if (row < g.m && left > 0) {
            const float sa = g.sa[row];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(sum[e], sa, e < left ? g.sb[col + e] : 0.0f);
            store4(c + row * g.ldc + col, left < 4 ? (int)left : 4, v, g.wide);
        }
    }
}

template <class T, int NT, int MT, int WS>
hipError_t launch_few(const Args& g, T* c, hipStream_t stream) {
    const dim3 grid((unsigned)((g.n + NT * 16 - 1) / (NT * 16)), (unsigned)((g.m + MT * 16 - 1) / (MT * 16)));
    hipLaunchKernelGGL((k_mm_int8_few<T, NT, MT, WS>), grid, dim3(WS * WAVE), 0, stream, g, c);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const Args& g, T* c, hipStream_t stream) {
    if (g.m <= 16) return launch_few<T, 1, 1, 16>(g, c, stream);
    if (g.m <= 32) return launch_few<T, 1, 2, 8>(g, c, stream);
    if (g.m <= 64) return launch_few<T, 2, 4, 8>(g, c, stream);
    const auto tiles = [&](int64_t bn, int64_t bm) { return ((g.n + bn - 1) / bn) * ((g.m + bm - 1) / bm); };
    if (tiles(256, 256) >= 192) return launch_pipe<T, 256, 256, 2, 4>(g, c, stream);
    if (tiles(128, 128) >= 192) return launch_pipe<T, 128, 128, 2, 2>(g, c, stream);
    return launch_tile<T, 64, 64, 2, 2>(g, c, stream);
}

}  // namespace

hipError_t launch_matmul_int8(const void* a, const float* a_scale, int64_t lda, const void* b, const float* b_scale,
                              int64_t ldb, int64_t m, int64_t n, int64_t k, void* c, bool bf16, int64_t ldc,
                              hipStream_t stream) {
    const Args g{static_cast<const uint8_t*>(a), a_scale, lda, static_cast<const uint8_t*>(b), b_scale, ldb, m, n,
                 (int32_t)k, ldc, ldc % 4 == 0 && reinterpret_cast<uintptr_t>(c) % (bf16 ? 8 : 16) == 0};
    return bf16 ? launch(g, static_cast<BF16*>(c), stream) : launch(g, static_cast<float*>(c), stream);
}

}  // namespace qc
