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
    __device__ __forceinline__ void init(const uint8_t* mat, int64_t ld, int64_t row0, int64_t rows, int padded) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
        const int lrow = lane_id() >> 3, piece = (lane_id() & 7) ^ lrow;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = min((wave_id() * N + i) * 8 + lrow, last) * (int)ld + piece * 16;
        rsrc = buffer_of(mat + row0 * ld, last * (int)ld + padded);
    }
    // `over`: how far this lane's piece at k0 lies past the last one of the row
    __device__ __forceinline__ void load(uint32_t lds, int k0, int over) const {
#pragma unroll
        for (int i = 0; i < N; ++i) load_lds16(rsrc, lds + (wave_id() * N + i) * 1024, off[i] - over, k0);
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
    const int wn = wave_id() % WN, wm = wave_id() / WN;
    const int l = lane_id();

    const int padded = (g.k + 15) & ~15;
    Loader<BN, NW> lb;
    Loader<BM, NW> la;
    lb.init(g.b, g.ldb, n0, g.n, padded);
    la.init(g.a, g.lda, m0, g.m, padded);
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
        lb.load(lds0 + buf * TILE, t * BK, over);
        la.load(lds0 + buf * TILE + TB, t * BK, over);
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
// 64 bytes of k.  Four stages lie in LDS: one is read, the next has landed,
// two are on their way, so a load has two stages' time to arrive.  A wave
// reads its fragments ahead of their use, into the next stage too: the wait
// for that one, and the only barrier, stand in the middle of a stage, where
// the fragments already read keep the matrix cores busy across it.
//
// Rows are 64 bytes in LDS, piece c of row r in slot c ^ ((r >> 1) & 3):
// conflict-free for the fragment reads (16 rows, 4 pieces).
constexpr int SK = 64;

template <int ROWS, int NW>
struct StageLoader {
    static constexpr int N = ROWS / 16 / NW;  // loads per wave: 16 rows each
    int off[N];
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ void init(const uint8_t* mat, int64_t ld, int64_t row0, int64_t rows, int padded,
                                         int piece, int wave) {
        const int64_t left = rows - 1 - row0;
        const int last = left < ROWS - 1 ? (int)left : ROWS - 1;
#pragma unroll
        for (int i = 0; i < N; ++i)
            off[i] = min((wave * N + i) * 16 + (lane_id() >> 2), last) * (int)ld + piece * 16;
        rsrc = buffer_of(mat + row0 * ld, last * (int)ld + padded);
    }
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, int k0, int over) const {
        load_lds16(rsrc, lds + (wave * N + i) * 1024, off[i] - over, k0);
    }
};

template <int ROWS, int THREADS>
__device__ __forceinline__ void zero_stage_tail(uint8_t* lds, int valid) {
    for (int i = threadIdx.x; i < ROWS * 4; i += THREADS) {
        const int r = i >> 2, c = i & 3;
        uint32_t* p = reinterpret_cast<uint32_t*>(lds + r * SK + ((c ^ ((r >> 1) & 3)) << 4));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int keep = valid - (c * 16 + w * 4);  // bytes of this word that stay
            if (keep <= 0) p[w] = 0u;
            else if (keep < 4) p[w] &= (1u << (8 * keep)) - 1u;
        }
    }
}

template <class T, int BN, int BM, int WN, int WM>
__global__ void __launch_bounds__(WN * WM * WAVE)
k_mm_int8_pipe(Args g, T* __restrict__ c) {
    constexpr int NW = WN * WM, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FM = BM / WM / 16;
    constexpr int AHEAD = FN >= 8 ? 3 : 2;           // weight fragments read ahead (of a ring of 4)
    constexpr int TB = BN * SK, STAGE = (BN + BM) * SK;  // weights first, then tokens
    constexpr int LOADS = (BN + BM) / 16 / NW;
    static_assert(FN % 4 == 0 && FM % (FN / 2) == 0 && LOADS % (FN / 2) == 0, "fragment schedule");
    __shared__ __align__(1024) uint8_t lds[4 * STAGE];

    const uint32_t tn = (uint32_t)((g.n + BN - 1) / BN), tm = (uint32_t)((g.m + BM - 1) / BM);
    const Tile2 tile = tile_of<4>(blockIdx.x, tn, tm);
    const int64_t n0 = (int64_t)tile.x * BN, m0 = (int64_t)tile.y * BM;
    const int w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wm = w / WN;
    const int l = lane_id();
    const int padded = (g.k + 15) & ~15;
    const int piece = (l & 3) ^ ((l >> 3) & 3);  // of row l / 4
    StageLoader<BN, NW> lb;
    StageLoader<BM, NW> la;
    lb.init(g.b, g.ldb, n0, g.n, padded, piece, w);
    la.init(g.a, g.lda, m0, g.m, padded, piece, w);

    const int stages = (g.k + 2 * SK - 1) / (2 * SK) * 2;  // an even number; the last may be all zeros
    const int whole = g.k / SK;                            // stages from here on hold bytes past k
    const uint32_t lds0 = lds_addr(lds);
    // load `part` (of LOADS) of stage s; `over` is how far a lane's piece lies past the last one of its row
    auto fetch_part = [&](int part, int s, int over) {
        const uint32_t at = lds0 + (s & 3) * STAGE;
        const int k0 = min(s * SK, padded - 16);
        if (part < lb.N) lb.load(part, at, w, k0, over);
        else la.load(part - lb.N, at + TB, w, k0, over);
    };
    auto over_of = [&](int s) { return max(min(s * SK, padded - 16) + piece * 16 - (padded - 16), 0); };
    auto fetch = [&](int s) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) fetch_part(part, s, over_of(s));
    };
    auto cut = [&](int s) {
        if (s >= whole && s < stages) {  // the weights' bytes past k become zeros (integers: one side is enough)
            zero_stage_tail<BN, THREADS>(lds + (s & 3) * STAGE, max(g.k - s * SK, 0));
            __syncthreads();
        }
    };

    const int frag = (l & 15) * SK + (((l >> 4) ^ ((l >> 1) & 3)) << 4);
    const int rb = wn * FN * 1024 + frag, ra = TB + wm * FM * 1024 + frag;
    // s: the stage's buffer, 0 to 3
    auto read_b = [&](int s, int i) { return *reinterpret_cast<const i32x4*>(lds + s * STAGE + rb + i * 1024); };
    auto read_a = [&](int s, int j) { return *reinterpret_cast<const i32x4*>(lds + s * STAGE + ra + j * 1024); };

    i32x4 acc[FN][FM] = {};
    i32x4 fb[4], fa[2][FM];
    // Stage s, s = PH modulo 4 (PH modulo 2 where it is not FAST).  FAST: stage
    // s + 3 exists and s + 1 is whole.  A load is issued with each fragment
    // after the barrier: all of them at once would hold up the waves.
    auto stage = [&](auto phase, auto fast, int s) {
        constexpr int PH = decltype(phase)::value, P = PH & 1;
        constexpr bool FAST = decltype(fast)::value;
        const int here = FAST ? PH : s & 3, next = FAST ? (PH + 1) & 3 : (s + 1) & 3;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            if (i == FN / 2) {
                if (FAST || s + 2 < stages) lds_landed_but<LOADS>();
                else lds_landed();
                if (!FAST) cut(s + 1);
            }
            fb[(i + AHEAD) % 4] = i + AHEAD < FN ? read_b(here, i + AHEAD) : read_b(next, i + AHEAD - FN);
            if (i >= FN / 2) {
                constexpr int E = FM / (FN / 2), D = LOADS / (FN / 2);
#pragma unroll
                for (int e = 0; e < E; ++e) fa[P ^ 1][(i - FN / 2) * E + e] = read_a(next, (i - FN / 2) * E + e);
                // over the stage that every wave has left
                if (FAST || s + 3 < stages) {
#pragma unroll
                    for (int d = 0; d < D; ++d) fetch_part((i - FN / 2) * D + d, s + 3, FAST ? 0 : over_of(s + 3));
                }
            }
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i % 4], fa[P][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
        }
    };
    using std::integral_constant;

    fetch(0);
    fetch(1);
    if (stages > 2) {
        fetch(2);
        lds_landed_but<2 * LOADS>();
    } else {
        lds_landed_but<LOADS>();
    }
    cut(0);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[0][j] = read_a(0, j);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fb[i] = read_b(0, i);
    int s = 0;
    for (; s + 6 < min(stages, whole); s += 4) {
        stage(integral_constant<int, 0>{}, std::true_type{}, s);
        stage(integral_constant<int, 1>{}, std::true_type{}, s + 1);
        stage(integral_constant<int, 2>{}, std::true_type{}, s + 2);
        stage(integral_constant<int, 3>{}, std::true_type{}, s + 3);
    }
#pragma unroll 1
    for (; s < stages; s += 2) {
        stage(integral_constant<int, 0>{}, std::false_type{}, s);
        stage(integral_constant<int, 1>{}, std::false_type{}, s + 1);
    }

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
            const int at = ch * BK + (l >> 4) * 32 + h * 16;
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
                    const int keep = g.k - (ch * BK + (l >> 4) * 32 + h * 16 + e * 4);
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
