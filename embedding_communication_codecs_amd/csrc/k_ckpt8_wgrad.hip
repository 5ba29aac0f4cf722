// k_ckpt8_wgrad.hip -- the weight gradient of a linear layer whose input was
// kept in 8 bits: dW[n][d] (+)= sum over tokens t of dY[t][n] * X[t][d], X the
// values a checkpoint holds (codes times a power of two per 32 channels).
//
// X's values are exact in bf16, so they go to v_mfma_f32_16x16x32_bf16 as
// they are and every product is exact in fp32: nothing is rounded but the
// fp32 sums.  A bf16 dY goes in as it is too; an fp32 dY as three bf16
// pieces of 8 mantissa bits each, which add up to it exactly; bits of it that
// are too small for a bf16 value are added afterwards (add_rest).
//
// Both operands are summed over their slow axis.  Tiles of 32 tokens (64 in
// the simple kernel) lie in LDS as [token][channel] and are read with
// ds_read_b64_tr_b16, which hands each lane four tokens of one channel.
//
// 16384 x 4096 x 8192 (tokens, n, dim) takes 830-900 us, 1.22-1.33 PFLOP/s,
// and 4096 x 4096 x 4096 116-122 us, 1.15, where the matrix cores alone run at
// 1.85-1.97 PFLOP/s on random bf16 values.  They are busy 0.60 of the cycles:
// a stage's barrier, fragment reads and conversion leave them waiting for the
// rest.  Power takes the smaller part of the difference (all zeros take 747
// and 105 us).  Where the conversion and the reads stand among the products,
// and the waves' priorities, do not change these by more than 2%.
//
// Tiles of 128 x 128 are bound by their stages' latency: 0.45-0.55 us for 0.11 us
// of products, with one wave a SIMD and loads that run three stages ahead
// (2048 x 2048 x 2048: 64 stages, 34 us, matrix cores busy 0.22).  Splits that
// are joined take a second launch of 4 to 5 us.
#include "qc_lds.hpp"
#include "qc_launch.hpp"

#include <type_traits>

namespace qc {
namespace {

typedef __attribute__((address_space(3))) s16x4* lds4;
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));  // four values of dW, wherever they start
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

struct Args {
    const void* dy;
    int64_t ldy;
    const uint8_t* codes;
    const uint8_t* exps;
    int64_t pitch, epitch;
    int64_t rows, n, dim;
    int64_t rows_per_split;  // a multiple of the token tile
    void* out;               // dW, or the first split's partial sums
    int64_t ldw, split_stride;
    int32_t out_bf16, accumulate;
};

// Byte offset of 16-byte piece `c` of token `t` in a tile of `row_bytes` a
// token.  A fragment read takes 32 bytes of each of 16 tokens; the xor puts
// eight neighbouring tokens on different banks.
__device__ __forceinline__ int place(int t, int c, int row_bytes) { return t * row_bytes + ((c ^ (2 * (t & 7))) << 4); }

// Four bf16 values from four codes: code * step is exact and its upper half
// is the bf16 value.
__device__ __forceinline__ u32x2 held4(uint32_t word, float step) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(code_of(word, i) * step);
    return u32x2{__builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
}

// The three pieces of an fp32 value (8 mantissa bits each, cut off, so their
// sum is exact); an infinity or a NaN is its first piece alone.  `lost`
// gathers the bits that the third leaves (its lower 16).
__device__ __forceinline__ void pieces(float x, uint32_t (&p)[3], uint32_t& lost) {
    const uint32_t b = __float_as_uint(x);
    if ((b & kInfBits) == kInfBits) {
        p[0] = bf16_bits(x);
        p[1] = p[2] = 0;
        return;
    }
    const float r = x - __uint_as_float(b & 0xFFFF0000u);
    const uint32_t rb = __float_as_uint(r);
    p[0] = b >> 16;
    p[1] = rb >> 16;
    const uint32_t last = __float_as_uint(r - __uint_as_float(rb & 0xFFFF0000u));
    p[2] = last >> 16;
    lost |= last;
}

// What the three pieces leave of an fp32 gradient: bf16 has no bits below
// 2^-133, so where a gradient below 2^-110 has some, no piece takes them.
__device__ __forceinline__ float rest_of(float x) {
    if ((__float_as_uint(x) & kInfBits) == kInfBits) return 0.0f;
#pragma unroll
    for (int i = 0; i < 3; ++i) x -= __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    return x;
}

// Whether such remainders can change a wave's sums (their layout: store_dw):
// a product of one is below 2^-133 * 127 steps, and leaves a sum of 2^26 times
// that and more as it is, being less than a quarter of its step.  The steps
// are those of the wave's channels; a NaN group's sums are NaN whatever is
// added.
template <int FN, int FD>
__device__ __forceinline__ bool rest_matters(const Args& g, const f32x4 (&acc)[FD][FN], int64_t n0, int64_t d0,
                                             int64_t t_first, int64_t t_end) {
    constexpr int U = 8, GROUPS = FD / 2;
    const int l = lane_id();
    uint32_t most = 0;
    for (int64_t t0 = t_first + l; t0 - l < t_end; t0 += U * WAVE) {
        uint32_t byte[U][GROUPS];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < GROUPS; ++k)
                byte[u][k] = g.exps[min(t0 + u * WAVE, t_end - 1) * g.epitch + min(d0 / 32 + k, g.epitch - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) most = umax(most, byte[u][k] == kCkptNaN ? 0u : byte[u][k]);
    }
    const float large = ckpt_step(group_max_u32<WAVE>(most)) * (127.0f * 0x1p-107f);
    bool small = false;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FD; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                small |= fabsf(acc[i][j][e]) < large && n0 + j * 16 + (l & 15) < g.n &&
                         d0 + 16 * i + 4 * (l >> 4) + e < g.dim;
    return __any(small);
}

// Adds those remainders' products to a wave's sums in fp32 multiply-adds; a
// remainder has 16 bits and X 8, so the products are exact.  Only where they
// matter: the wave looks for its tokens that have a remainder among its
// channels, a token for 16 lanes, and multiplies for those, four at a time.
// 4096 x 4096 x 4096 of normal gradients 347 us (344 without the look at their
// bits); some of them, few or many, at 1e-36 400, for finding that they do not
// matter; with sums as small as they are, 650 for one in a million, 1,230 for
// one in a thousand and 5,600 for every other.
template <int FN, int FD>
__device__ __forceinline__ void add_rest(const Args& g, f32x4 (&acc)[FD][FN], int64_t n0, int64_t d0, int64_t t_first,
                                         int64_t t_end) {
    constexpr uint32_t kBelow = (127u - 110u) << 24;  // 2^-110's bits, shifted as below
    const int l = lane_id();
    const float* column[FN];  // this lane's channels; those past n repeat the last one (sums that are not stored)
#pragma unroll
    for (int j = 0; j < FN; ++j)
        column[j] = static_cast<const float*>(g.dy) + min(n0 + j * 16 + (l & 15), g.n - 1);
    auto gradient = [&](int64_t t, int j) {
        const float x = column[j][min(t, t_end - 1) * g.ldy];  // without a branch: the loads are on their way together
        return t < t_end ? x : 0.0f;
    };
    for (int64_t t0 = t_first; t0 < t_end; t0 += 32) {
        bool small[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            uint32_t least = ~0u;  // of the magnitudes' bits less one: zeros are the largest
#pragma unroll
            for (int j = 0; j < FN; ++j)
                least = min(least, (__float_as_uint(gradient(t0 + 4 * u + (l >> 4), j)) << 1) - 1u);
            small[u] = least < kBelow;
        }
        uint32_t tokens = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint64_t lanes = __ballot(small[u]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tokens |= (lanes >> (16 * q) & 0xFFFFu) ? 1u << (4 * u + q) : 0u;
        }
        while (tokens) {
            float r[4][FN], step[4][FD];
            uint32_t word[4][FD];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // none left: a token past the end, whose gradients read as zeros
                const int64_t t = tokens ? t0 + __ffs((int)tokens) - 1 : t_end;
                tokens &= tokens - 1u;
#pragma unroll
                for (int j = 0; j < FN; ++j) r[u][j] = gradient(t, j);
#pragma unroll
                for (int i = 0; i < FD; ++i) {
                    // past the row: sums that are not stored
                    const int64_t tx = min(t, t_end - 1), d = min(d0 + 16 * i + 4 * (l >> 4), g.pitch - 4);
                    word[u][i] = *reinterpret_cast<const uint32_t*>(g.codes + tx * g.pitch + d);
                    step[u][i] = ckpt_step(g.exps[tx * g.epitch + d / 32]);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int j = 0; j < FN; ++j) r[u][j] = rest_of(r[u][j]);
#pragma unroll
                for (int i = 0; i < FD; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = code_of(word[u][i], e) * step[u][i];
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j][e] = __builtin_fmaf(r[u][j], x, acc[i][j][e]);
                    }
            }
        }
    }
}

// A wave's sums to dW.  Lane l holds output channel l % 16 of each of FN
// tiles, input channels 4 * (l / 16) .. + 3 of each of FD.  Four of them are
// one store wherever their row starts (1000 x 4096 x 4095 46 us against 69 with
// a store a value).
template <int FN, int FD>
__device__ __forceinline__ void store_dw(const Args& g, f32x4 (&acc)[FD][FN], int64_t n0, int64_t d0) {
    const int l = lane_id();
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int64_t n = n0 + j * 16 + (l & 15);
        if (n >= g.n) continue;
        const int64_t d = d0 + 4 * (l >> 4);
        if (g.out_bf16) {
            BF16* o = static_cast<BF16*>(g.out) + n * g.ldw + d;
#pragma unroll
            for (int i = 0; i < FD; ++i) {
                const int64_t left = g.dim - d - 16 * i;
                const f32x4 v = acc[i][j];
                if (left >= 4)
                    *reinterpret_cast<u32x2_a2*>(o + 16 * i) = u32x2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
                else
                    for (int e = 0; e < 4; ++e)
                        if (e < left) put(o + 16 * i + e, v[e]);
            }
            continue;
        }
        float* o = static_cast<float*>(g.out) + (int64_t)blockIdx.y * g.split_stride + n * g.ldw + d;
        if (g.accumulate) {  // what is there, all of it before the first store
#pragma unroll
            for (int i = 0; i < FD; ++i) {
                const int64_t left = g.dim - d - 16 * i;
                if (left >= 4) acc[i][j] += *reinterpret_cast<const f32x4_a4*>(o + 16 * i);
                else
                    for (int e = 0; e < 4; ++e)
                        if (e < left) acc[i][j][e] += o[16 * i + e];
            }
        }
#pragma unroll
        for (int i = 0; i < FD; ++i) {
            const int64_t left = g.dim - d - 16 * i;
            if (left >= 4) *reinterpret_cast<f32x4_a4*>(o + 16 * i) = acc[i][j];
            else
                for (int e = 0; e < 4; ++e)
                    if (e < left) o[16 * i + e] = acc[i][j][e];
        }
    }
}

// ------------------------------------------------------------------- simple
// Gradients of very few channels (n below 8 in bf16, below 4 in fp32), as the
// output layer of a regression, a reward or a few classes has them, whose rows
// may be shorter than one load of the kernels below.  One block: BN output
// channels (columns of dY) x BD input channels (columns of X), WN x WD waves,
// TK tokens a step, two steps in LDS; both operands pass through registers.
// P: pieces of dY (1: bf16, 3: fp32).
template <int P, int BN, int BD, int WN, int WD, int TK>
__global__ void __launch_bounds__(WN * WD * WAVE)
k_ckpt8_wgrad(Args g) {
    constexpr int NW = WN * WD, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FD = BD / WD / 16;
    constexpr int YB = BN * 2, XB = BD * 2;      // bytes of a token in a tile
    constexpr int YT = TK * YB, XT = TK * XB;    // bytes of a tile
    constexpr int TILE = P * YT + XT;            // pieces of dY first, then X
    constexpr int XG = TK * BD / 32 / THREADS;   // groups of X a thread converts
    static_assert(XG >= 1, "a group for every thread");
    __shared__ __align__(1024) uint8_t lds[2 * TILE];
    __shared__ int rest;  // some gradient of the block has more bits than its pieces

    const int64_t tn = (g.n + BN - 1) / BN;
    const int64_t n0 = ((int64_t)blockIdx.x % tn) * BN, d0 = ((int64_t)blockIdx.x / tn) * BD;
    const int64_t t_first = (int64_t)blockIdx.y * g.rows_per_split;
    const int64_t t_end = min(g.rows, t_first + g.rows_per_split);
    const int l = lane_id(), w = wave_id();
    const int wn = w % WN, wd = w / WN;

    f32x4 acc[FD][FN] = {};

    // ---- X: codes and steps of this thread's groups, then bf16 into LDS
    u32x4 xw[XG][2];
    float xstep[XG];
    auto x_get = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < XG; ++i) {
            const int id = i * THREADS + threadIdx.x;
            const int64_t t = t0 + id / (BD / 32);
            const int64_t d = d0 + (id % (BD / 32)) * 32;
            const bool in = t < t_end && d < g.dim;
            xw[i][0] = xw[i][1] = u32x4{0, 0, 0, 0};
            xstep[i] = 0.0f;
            if (in) {
                const uint8_t* p = g.codes + t * g.pitch + d;
                xw[i][0] = ld_u4(p);
                xw[i][1] = ld_u4(p + 16);
                xstep[i] = ckpt_step(g.exps[t * g.epitch + d / 32]);
            }
        }
    };
    auto x_put = [&](uint8_t* tile) {
#pragma unroll
        for (int i = 0; i < XG; ++i) {
            const int id = i * THREADS + threadIdx.x;
            const int t = id / (BD / 32), c = (id % (BD / 32)) * 4;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const u32x2 a = held4(xw[i][h >> 1][2 * (h & 1)], xstep[i]);
                const u32x2 b = held4(xw[i][h >> 1][2 * (h & 1) + 1], xstep[i]);
                *reinterpret_cast<u32x4*>(tile + place(t, c + h, XB)) = u32x4{a.x, a.y, b.x, b.y};
            }
        }
    };

    // ---- dY
    constexpr int YC = TK * BN / 8 / THREADS;  // pieces of 8 values a thread stages
    float yv[YC][8];
    uint32_t lost = 0;
    auto y_get = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < YC; ++i) {
            const int id = i * THREADS + threadIdx.x;
            const int64_t t = t0 + id / (BN / 8), col = n0 + (id % (BN / 8)) * 8;
            const int64_t left = t < t_end ? g.n - col : 0;
            if constexpr (P == 1) load8(static_cast<const BF16*>(g.dy) + t * g.ldy + col, left, yv[i]);
            else load8(static_cast<const float*>(g.dy) + t * g.ldy + col, left, yv[i]);
        }
    };
    auto y_put = [&](uint8_t* tile) {
#pragma unroll
        for (int i = 0; i < YC; ++i) {
            const int id = i * THREADS + threadIdx.x;
            const int at = place(id / (BN / 8), id % (BN / 8), YB);
            uint32_t o[P][4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if constexpr (P == 1) {  // bf16 values again: exact
                    o[0][h] = (__float_as_uint(yv[i][2 * h]) >> 16) | (__float_as_uint(yv[i][2 * h + 1]) & 0xFFFF0000u);
                } else {
                    uint32_t a[3], b[3];
                    pieces(yv[i][2 * h], a, lost);
                    pieces(yv[i][2 * h + 1], b, lost);
#pragma unroll
                    for (int q = 0; q < P; ++q) o[q][h] = a[q] | (b[q] << 16);
                }
            }
#pragma unroll
            for (int q = 0; q < P; ++q)
                *reinterpret_cast<u32x4*>(tile + q * YT + at) = u32x4{o[q][0], o[q][1], o[q][2], o[q][3]};
        }
        if (P == 3 && (lost & 0xFFFFu)) rest = 1;
    };

    // ---- fragments: lane l reads 8 bytes of token r*16 + l/4, 16 channels
    // by four lanes, and gets four tokens of channel l % 16
    const int ft = l >> 2;  // 0..15
    auto frag = [&](const uint8_t* tile, int row_bytes, int f, int kk) {
        const int c = f * 2 + ((l & 3) >> 1);
        s16x4 p[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
            p[r] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds4)(tile + place(kk * 32 + r * 16 + ft, c, row_bytes) + 8 * (l & 1)));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, s16x8{p[0].x, p[0].y, p[0].z, p[0].w, p[1].x, p[1].y, p[1].z, p[1].w});
    };
    auto compute = [&](const uint8_t* tile) {
#pragma unroll
        for (int kk = 0; kk < TK / 32; ++kk) {
            bf16x8 fx[FD];
#pragma unroll
            for (int i = 0; i < FD; ++i) fx[i] = frag(tile + P * YT, XB, wd * FD + i, kk);
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const bf16x8 fy = frag(tile + q * YT, YB, wn * FN + j, kk);
#pragma unroll
                    for (int i = 0; i < FD; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[i], fy, acc[i][j], 0, 0, 0);
                }
        }
    };

    if (t_first < t_end) {
        y_get(t_first);
        if (P == 3) {
            if (threadIdx.x == 0) rest = 0;
            __syncthreads();
        }
        y_put(lds);
        x_get(t_first);
        x_put(lds + P * YT);
        int buf = 0;
        for (int64_t t0 = t_first; t0 < t_end; t0 += TK, buf ^= 1) {
            __syncthreads();
            const bool more = t0 + TK < t_end;
            if (more) {
                x_get(t0 + TK);
                y_get(t0 + TK);
            }
            compute(lds + buf * TILE);
            if (more) {
                x_put(lds + (buf ^ 1) * TILE + P * YT);
                y_put(lds + (buf ^ 1) * TILE);
            }
        }
        // set before the last barrier, if at all
        if (P == 3 && rest) {
            const int64_t nw = n0 + wn * FN * 16, dw = d0 + wd * FD * 16;
            if (rest_matters<FN, FD>(g, acc, nw, dw, t_first, t_end)) add_rest<FN, FD>(g, acc, nw, dw, t_first, t_end);
        }
    }

    store_dw<FN, FD>(g, acc, n0 + wn * FN * 16, d0 + wd * FD * 16);
}

// As pieces, of four neighbours, packed (word 0 holds values 0 and 1), without
// a branch.
__device__ __forceinline__ void pieces4(f32x4 x, u32x2 (&q)[3], uint32_t& lost) {
    auto upper = [](uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); };
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i == 0) {
                x[e] = __builtin_canonicalizef(x[e]);  // a NaN's upper half is a NaN then
            } else {
                const float r = x[e] - __uint_as_float(b[e] & 0xFFFF0000u);
                x[e] = i > 1 || __builtin_isfinite(x[e]) ? r : 0.0f;  // an infinity is its first piece alone
            }
            b[e] = __float_as_uint(x[e]);
            if (i == 2) lost |= b[e];
        }
        q[i] = u32x2{upper(b[0], b[1]), upper(b[2], b[3])};
    }
}

// --------------------------------------------------------------- pipelined
// bf16 gradients, n at least 8.  One block computes BN output x BD input
// channels with WN x WD waves, in stages of 32 tokens.  Everything is loaded
// straight into LDS, two stages before its use: dY as it is, X as codes and
// exponent words.  Each lane's 16 codes and their exponents land in a place of
// its own, so the lane converts them to bf16 as soon as its own wave's loads
// have landed and writes them to X's tile, which the next barrier shows to the
// block.  Load batch b holds dY of stage b and X of stage b + 1: converted X is
// needed one barrier later than landed dY.
//
// As in the INT8 product, fragments are read ahead of their use and into
// the next stage, and the only barrier of a stage stands in its middle.
constexpr int ST = 32;  // tokens of a stage
// Bytes a descriptor reaches from its stage's first row.  A stage's offsets stay
// below 2^31 (32 rows at most 2^25 bytes apart); a negative one counts as 2^31 and
// more, past the descriptor, and loads zeros.  Descriptors that end where the
// matrix does cost scalar registers and 3 to 10% where stages are few (515 x 8 x
// 300: 9.0 us against 8.3), so that no load passes a matrix' end rests on the
// clamps below alone.
constexpr int kReach = 0x7FFFFFFF;

template <int BN, int BD, int WN, int WD>
__global__ void __launch_bounds__(WN * WD * WAVE)
k_ckpt8_wgrad_pipe(Args g) {
    constexpr int NW = WN * WD, THREADS = NW * WAVE;
    constexpr int FN = BN / WN / 16, FD = BD / WD / 16;
    constexpr int AHEAD = 2;  // fragments of dY read ahead (of a ring of 4)
    constexpr int YB = BN * 2, XB = BD * 2;        // bytes of a token in a tile
    constexpr int YT = ST * YB, XT = ST * XB;
    constexpr int YN = YT / 1024 / NW;             // loads of dY a wave and stage
    constexpr int LOADS = YN + 2;                  // and X's codes and exponents
    constexpr int TPW = 1024 / BD;                 // tokens of X a wave loads
    constexpr int RAW = 1024 + 256;                // a wave's codes and exponents of a stage
    static_assert(TPW * NW == ST && FN % 4 == 0 && YN >= 1, "tile shape");
    constexpr int XAT = 4 * YT, RAT = XAT + 2 * XT;  // LDS: four dY tiles, two X tiles, four raw stages
    __shared__ __align__(1024) uint8_t lds[RAT + 4 * NW * RAW];

    const uint32_t tn = (uint32_t)((g.n + BN - 1) / BN), td = (uint32_t)((g.dim + BD - 1) / BD);
    const Tile2 tile = tile_of<8>(blockIdx.x, tn, td);
    const int64_t n0 = (int64_t)tile.x * BN, d0 = (int64_t)tile.y * BD;
    const int64_t t_first = (int64_t)blockIdx.y * g.rows_per_split;
    const int64_t tokens = min(g.rows - t_first, g.rows_per_split);
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wd = w / WN;

    const int stages = (int)((tokens + 2 * ST - 1) / (2 * ST)) * 2;  // even; the last may have no token
    const int whole = (int)(tokens / ST);
    const uint32_t lds0 = lds_addr(lds);

    // ---- loads, of 16 bytes a lane at any alignment of dY's rows.  Tokens past
    // the end repeat the last one and are zeroed in LDS; pieces past a row's
    // end repeat its last piece (their sums are not stored).  A row's last
    // piece may reach past n: into the next row, whose values fall on columns
    // that are not stored.  The matrix's last row has no next one: there the
    // piece is taken from n - 8, and cut() puts its values in their places.
    const uint8_t* ybase = static_cast<const uint8_t*>(g.dy) + t_first * g.ldy * 2;  // column 0: offsets stay positive
    const uint8_t* xbase = g.codes + t_first * g.pitch;
    const uint8_t* ebase = g.exps + t_first * g.epitch;
    const int64_t last_piece = (g.n - 1) / 8 * 8;
    const bool patch = t_first + tokens == g.rows && g.n % 8 != 0;
    const int first_col = (int)n0, last_col = (int)last_piece;
    auto ytok = [&](int i, int lane) { return (w * YN + i) * (1024 / YB) + lane / (YB / 16); };
    auto ycol = [&](int i, int lane) {
        const int c = (lane % (YB / 16)) ^ (2 * (ytok(i, lane) & 7));
        return min(first_col + c * 8, last_col);
    };
    int yoff[YN];
#pragma unroll
    for (int i = 0; i < YN; ++i) yoff[i] = (ytok(i, l) * (int)g.ldy + ycol(i, l)) * 2;
    const int xt = w * TPW + l / (BD / 16), xq = l % (BD / 16);  // this lane's token of a stage, and 16 codes of it
    const int xcol = (int)min(d0 + xq * 16, g.pitch - 16);
    const int ecol = (int)min((d0 + xq * 16) / 128 * 4, g.epitch - 4);
    auto y_load = [&](auto fast, int i, int s) {
        int64_t t0 = (int64_t)s * ST;
        int off = yoff[i];
        if (!decltype(fast)::value) {
            t0 = min(t0, tokens - 1);
            int lane = l;
            asm("" : "+v"(lane));  // computed anew: held through the main loop, these would not fit the registers
            const int last = (int)min(tokens - 1 - t0, (int64_t)ST), t = min(ytok(i, lane), last);
            const int col = ycol(i, lane);
            off = (t * (int)g.ldy + (patch && t == last && col == last_col ? (int)g.n - 8 : col)) * 2;
        }
        load_lds16(buffer_of(ybase + t0 * g.ldy * 2, kReach), lds0 + (s & 3) * YT + (w * YN + i) * 1024, off, 0);
    };
    auto x_load = [&](auto fast, int part, int s) {
        int64_t t0 = (int64_t)s * ST;
        int t = xt;
        if (!decltype(fast)::value) {
            t0 = min(t0, tokens - 1);
            t = min(xt, (int)min(tokens - 1 - t0, (int64_t)ST));
        }
        const uint32_t at = lds0 + RAT + ((s & 3) * NW + w) * RAW;
        if (part == 0) load_lds16(buffer_of(xbase + t0 * g.pitch, kReach), at, t * (int)g.pitch + xcol, 0);
        else load_lds4(buffer_of(ebase + t0 * g.epitch, kReach), at + 1024, t * (int)g.epitch + ecol, 0);
    };
    auto load = [&](auto fast, int part, int batch) {  // one of the LOADS of a batch
        if (part < YN) y_load(fast, part, batch);
        else x_load(fast, part - YN, batch + 1);
    };
    auto load_all = [&](int batch) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) load(std::false_type{}, part, batch);
    };

    // ---- X: this lane's codes of stage s to bf16
    u32x4 raw;
    uint32_t eword;
    auto x_read = [&](int s) {
        const uint8_t* at = lds + RAT + ((s & 3) * NW + w) * RAW;
        raw = *reinterpret_cast<const u32x4*>(at + l * 16);
        eword = *reinterpret_cast<const uint32_t*>(at + 1024 + l * 4);
    };
    // Of eight neighbouring lanes the upper four write their second piece
    // first: eight pieces of 16 bytes in different banks either time.
    const bool odd = (l & 4) != 0;
    const int xplace = place(xt, xq * 2 + odd, XB);
    auto x_put = [&](auto fast, int s) {
        float step = ckpt_step((eword >> (8 * ((xq >> 1) & 3))) & 0xFFu);
        u32x4 q = odd ? u32x4{raw.z, raw.w, raw.x, raw.y} : raw;
        if (!decltype(fast)::value && xt >= (int)min(tokens - (int64_t)s * ST, (int64_t)ST)) {
            step = 0.0f;
            q = u32x4{0, 0, 0, 0};
        }
        uint8_t* at = lds + XAT + (s & 1) * XT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x2 a = held4(q[2 * h], step), b = held4(q[2 * h + 1], step);
            *reinterpret_cast<u32x4*>(at + (xplace ^ (16 * h))) = u32x4{a.x, a.y, b.x, b.y};
        }
    };
    auto cut = [&](int s) {
        const bool last = patch && s == (int)((tokens - 1) / ST);
        if (!last && (s < whole || s >= stages)) return;
        // tokens past the end: zeros (X's are too, but an infinity times zero is not)
        uint8_t* at = lds + (s & 3) * YT;
        for (int i = (int)max(min(tokens - (int64_t)s * ST, (int64_t)ST), (int64_t)0) * YB + threadIdx.x * 16; i < YT;
             i += THREADS * 16)
            *reinterpret_cast<u32x4*>(at + i) = u32x4{0, 0, 0, 0};
        if (last && threadIdx.x < 8 && last_piece >= n0 && last_piece < n0 + BN) {
            const int64_t col = last_piece + threadIdx.x;
            const uint16_t v = col < g.n ? static_cast<const uint16_t*>(g.dy)[(g.rows - 1) * g.ldy + col] : 0;
            *reinterpret_cast<uint16_t*>(at + place((int)((tokens - 1) % ST), (int)(last_piece - n0) / 8, YB) +
                                         2 * threadIdx.x) = v;
        }
        __syncthreads();
    };

    // ---- fragments: lane l reads 8 bytes of token r * 16 + l / 4, and gets
    // four tokens of channel l % 16
    auto frag_at = [&](int f, int row_bytes) { return place(l >> 2, f * 2 + ((l & 3) >> 1), row_bytes) + 8 * (l & 1); };
    // FN and FD are powers of two up to 8: the other fragments are an xor away
    const int yf = frag_at(wn * FN, YB), xf = frag_at(wd * FD, XB);
    static_assert((FN & (FN - 1)) == 0 && FN <= 8 && (FD & (FD - 1)) == 0 && FD <= 8, "fragments");
    auto frag = [&](int at, int row_bytes) {
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds + at));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds + at + 16 * row_bytes));
        return __builtin_bit_cast(bf16x8, s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
    };
    auto read_y = [&](int buf, int j) { return frag(buf * YT + (yf ^ (j << 5)), YB); };
    auto read_x = [&](int buf, int i) { return frag(XAT + (buf & 1) * XT + (xf ^ (i << 5)), XB); };

    f32x4 acc[FD][FN] = {};
    bf16x8 fy[4], fx[2][FD];
    // Stage s, s = PH modulo 4 (PH modulo 2 where it is not FAST).  FAST: the
    // stages up to s + 4 are whole.
    auto stage = [&](auto phase, auto fast, int s) {
        constexpr int PH = decltype(phase)::value, P = PH & 1;
        constexpr bool FAST = decltype(fast)::value;
        const int here = FAST ? PH : s & 3, next = FAST ? (PH + 1) & 3 : (s + 1) & 3;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if (j == FN / 2) {
                if (FAST || s + 2 < stages) lds_landed_but<LOADS>();
                else lds_landed();
                if (!FAST) cut(s + 1);
                if (FAST || s + 2 < stages) x_read(s + 2);
            }
            fy[(j + AHEAD) % 4] = j + AHEAD < FN ? read_y(here, j + AHEAD) : read_y(next, j + AHEAD - FN);
            if (j >= FN / 2) {
                constexpr int H = FN / 2;  // this iteration's share of X's fragments and of the loads
#pragma unroll
                for (int e = (j - H) * FD / H; e < (j - H + 1) * FD / H; ++e) fx[P ^ 1][e] = read_x(next, e);
                // over what every wave has left
                if (FAST || s + 3 < stages) {
#pragma unroll
                    for (int d = (j - H) * LOADS / H; d < (j - H + 1) * LOADS / H; ++d) load(fast, d, s + 3);
                }
            }
            if (j == FN / 2 + 1 && (FAST || s + 2 < stages)) x_put(fast, s + 2);
#pragma unroll
            for (int i = 0; i < FD; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[P][i], fy[j % 4], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
        }
    };

    if (stages > 0) {  // an even number: two at least
        x_load(std::false_type{}, 0, 0);
        x_load(std::false_type{}, 1, 0);
        load_all(0);
        load_all(1);
        if (stages > 2) {
            load_all(2);
            lds_landed_but<2 * LOADS>();
        } else {
            lds_landed_but<LOADS>();
        }
        cut(0);
        x_read(0);
        x_put(std::false_type{}, 0);
        x_read(1);
        x_put(std::false_type{}, 1);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FD; ++i) fx[0][i] = read_x(0, i);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) fy[j] = read_y(0, j);
        using std::integral_constant;
        int s = 0;
        for (; s + 7 < whole; s += 4) {
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
    }
    store_dw<FN, FD>(g, acc, n0 + wn * FN * 16, d0 + wd * FD * 16);
}

// The same for fp32 gradients, n at least 4: each wave's part of dY lands in
// a place of its own too, and is taken apart into its three bf16 pieces, a
// tile each, when X is converted.  The three products of a step share X's
// fragments.
//
// A stage is three parts, a product with one piece of dY each, of FN steps.
// The barrier stands before the third part, whose fragments are in registers
// by then: every wave has read the stage's tiles, so the stage after next may
// be converted over them, and the next one is whole.  With the barrier and the
// first fragments at a stage's start, 4096 x 4096 x 4096 of normal values took
// 575 us; so it takes 340-380 with tiles of 128 x 256, three products at 1.08-1.2
// PFLOP/s.  128 x 128 reads and converts dY, the wider operand, twice as often
// for a product (494 us where 128 x 256 takes 347, values of few bits).
template <int BD>
__global__ void __launch_bounds__(512)
k_ckpt8_wgrad_pipe_f32(Args g) {
    constexpr int BN = 128, NW = 8, WN = 2, FN = 4, FD = BD / 64;
    constexpr int YB = BN * 2, XB = BD * 2, YT = ST * YB, XT = ST * XB;
    constexpr int YN = 2;                      // loads of dY a wave and stage
    constexpr int LOADS = YN + 2;              // and X's codes and exponents
    constexpr int TOK = 1024 / BD;             // tokens of X a wave loads
    constexpr int XW = ST / TOK;               // waves that load different ones
    constexpr int XH = BD / 128;               // pieces of 8 codes that a lane converts, of the 16 it loads
    constexpr int RAW = YN * 1024 + 1024 + 256;  // a wave's loads of a stage
    static_assert(YN * 1024 * NW == ST * BN * 4 && NW * WAVE * 8 * XH == ST * BD, "tile shape");
    constexpr int BUF = 3 * YT + XT, RAT = 2 * BUF;  // LDS: two buffers of tiles, three raw stages
    __shared__ __align__(1024) uint8_t lds[RAT + 3 * NW * RAW];
    __shared__ int rest;  // some gradient of the block has more bits than its pieces

    const uint32_t tn = (uint32_t)((g.n + BN - 1) / BN), td = (uint32_t)((g.dim + BD - 1) / BD);
    const Tile2 tile = tile_of<8>(blockIdx.x, tn, td);
    const int64_t n0 = (int64_t)tile.x * BN, d0 = (int64_t)tile.y * BD;
    const int64_t t_first = (int64_t)blockIdx.y * g.rows_per_split;
    const int64_t tokens = min(g.rows - t_first, g.rows_per_split);
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = w % WN, wd = w / WN;
    const int stages = (int)((tokens + ST - 1) / ST);
    const uint32_t lds0 = lds_addr(lds);

    // ---- loads: as above, with pieces of four values; the last row's short
    // piece is taken from n - 4 and moved up in registers
    const uint8_t* ybase = static_cast<const uint8_t*>(g.dy) + t_first * g.ldy * 4;
    const uint8_t* xbase = g.codes + t_first * g.pitch;
    const uint8_t* ebase = g.exps + t_first * g.epitch;
    const int64_t last_piece = (g.n - 1) / 4 * 4;
    const int yc = l & 31;                          // this lane's piece of a token
    const int ycol = (int)min(n0 + yc * 4, last_piece);
    const int yover = max(ycol + 4 - (int)g.n, 0);  // values of it past n
    auto token_y = [&](int i) { return (w * YN + i) * 2 + (l >> 5); };
    // this lane's token of a stage, and 16 codes of it
    const int xt = w % XW * TOK + l / (BD / 16), xq = l % (BD / 16);
    const int xcol = (int)min(d0 + xq * 16, g.pitch - 16);
    const int ecol = (int)min((d0 + xq * 16) / 128 * 4, g.epitch - 4);
    int yoff[YN];
#pragma unroll
    for (int i = 0; i < YN; ++i) yoff[i] = (token_y(i) * (int)g.ldy + ycol) * 4;
    const int xoff = xt * (int)g.pitch + xcol, eoff = xt * (int)g.epitch + ecol;
    // how many tokens a stage has (all of them but in the last one)
    auto tokens_of = [&](int s) { return (int)min(tokens - (int64_t)s * ST, (int64_t)ST); };
    // FAST, here and below: the stage is whole and not the matrix's last rows.
    // `slot`: the stage's number modulo 3.
    auto load = [&](auto fast, int part, int s, int slot) {  // one of the LOADS of a stage
        constexpr bool FAST = decltype(fast)::value;
        const int64_t t0 = (int64_t)s * ST;
        const int have = FAST ? ST : tokens_of(s);
        const uint32_t at = lds0 + RAT + (slot * NW + w) * RAW;
        if (part < YN) {
            int off = yoff[part];
            if (!FAST) {
                const int t = min(token_y(part), have - 1);
                off = (t * (int)g.ldy + ycol - (t_first + t0 + t == g.rows - 1 ? yover : 0)) * 4;
            }
            load_lds16(buffer_of(ybase + t0 * g.ldy * 4, kReach), at + part * 1024, off, 0);
        } else if (part == YN) {
            const int off = FAST ? xoff : min(xt, have - 1) * (int)g.pitch + xcol;
            load_lds16(buffer_of(xbase + t0 * g.pitch, kReach), at + YN * 1024, off, 0);
        } else {
            const int off = FAST ? eoff : min(xt, have - 1) * (int)g.epitch + ecol;
            load_lds4(buffer_of(ebase + t0 * g.epitch, kReach), at + YN * 1024 + 1024, off, 0);
        }
    };
    auto load_all = [&](int s) {
#pragma unroll
        for (int part = 0; part < LOADS; ++part) load(std::false_type{}, part, s, s % 3);
    };

    // ---- conversion of a stage by the wave that loaded it: of each load of
    // dY four values a lane, of X 8 * XH codes
    f32x4 raw_y[YN];
    u32x4 raw_x;
    uint32_t raw_e;
    auto read_raw = [&](int slot) {
        const uint8_t* at = lds + RAT + (slot * NW + w) * RAW;
#pragma unroll
        for (int i = 0; i < YN; ++i) raw_y[i] = *reinterpret_cast<const f32x4*>(at + i * 1024 + l * 16);
        raw_x = *reinterpret_cast<const u32x4*>(at + YN * 1024 + l * 16);
        raw_e = *reinterpret_cast<const uint32_t*>(at + YN * 1024 + 1024 + l * 4);
    };
    uint32_t lost = 0;
    auto convert_y = [&](auto fast, int i, int s, int buf) {
        f32x4 r = raw_y[i];
        const int t = token_y(i);
        if (!decltype(fast)::value) {  // tokens past the end, and the last row's short piece
            const int have = tokens_of(s);
            const int up = t_first + (int64_t)s * ST + t == g.rows - 1 ? yover : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = 0.0f;
#pragma unroll
                for (int f = e; f < 4; ++f)
                    if (f == e + up) v = r[f];
                r[e] = t < have ? v : 0.0f;
            }
        }
        u32x2 q[3];
        pieces4(r, q, lost);
        uint8_t* o = lds + buf * BUF + place(t, yc >> 1, YB) + 8 * (yc & 1);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x2*>(o + p * YT) = q[p];
    };
    // Where a lane has two pieces, the upper four of eight neighbouring lanes
    // write their second one first: eight pieces in different banks either
    // time.  Where it has one, the upper four waves have the second ones.
    const bool second = XH == 2 ? (l & 4) != 0 : w >= XW;
    const int xplace = place(xt, xq * 2 + second, XB);
    auto convert_x = [&](auto fast, int h, int s, int buf) {
        float step = ckpt_step((raw_e >> (8 * ((xq >> 1) & 3))) & 0xFFu);
        u32x2 q = second != (h == 1) ? u32x2{raw_x.z, raw_x.w} : u32x2{raw_x.x, raw_x.y};
        if (!decltype(fast)::value && xt >= tokens_of(s)) {
            step = 0.0f;
            q = u32x2{0, 0};
        }
        const u32x2 a = held4(q.x, step), b = held4(q.y, step);
        *reinterpret_cast<u32x4*>(lds + buf * BUF + 3 * YT + (xplace ^ (16 * h))) = u32x4{a.x, a.y, b.x, b.y};
    };

    auto frag_at = [&](int f, int row_bytes) { return place(l >> 2, f * 2 + ((l & 3) >> 1), row_bytes) + 8 * (l & 1); };
    const int yf = frag_at(wn * FN, YB), xf = 3 * YT + frag_at(wd * FD, XB);
    auto frag = [&](int at, int row_bytes) {
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds + at));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(lds + at + 16 * row_bytes));
        return __builtin_bit_cast(bf16x8, s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
    };
    auto read_y = [&](int buf, int p, int j) { return frag(buf * BUF + p * YT + (yf ^ (j << 5)), YB); };
    auto read_x = [&](int buf, int i) { return frag(buf * BUF + (xf ^ (i << 5)), XB); };

    f32x4 acc[FD][FN] = {};
    bf16x8 fx[2][FD], fy[2][FN];
    // Stage s, s = P modulo 2 and = rot modulo 3.  On entry its first
    // fragments and the raw values of stage s + 1 are in registers, and the
    // first part of dY's is converted.  FAST: the stages up to s + 4 are.
    auto stage = [&](auto phase, auto fast, int s, int rot) {
        constexpr int P = decltype(phase)::value;
        constexpr bool FAST = decltype(fast)::value;
        const int rot2 = rot == 0 ? 2 : rot - 1, rot1 = rot == 2 ? 0 : rot + 1;  // of s + 2; of s + 1 and s + 4
#pragma unroll
        for (int p = 0; p < 3; ++p) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if (p < 2) {
                    fy[(P + p + 1) & 1][j] = read_y(P, p + 1, j);
                    if (FAST || s + 1 < stages) {
                        if (p == 0 && j == 0) convert_y(fast, 1, s + 1, P ^ 1);
                        if (p == 0 && j == 2) convert_x(fast, 0, s + 1, P ^ 1);
                        if (p == 1 && j == 0 && XH == 2) convert_x(fast, 1, s + 1, P ^ 1);
                    }
                } else {
                    if (j == 0) {
                        // every gradient has been converted by the last stage
                        if (!FAST && s + 1 == stages && (lost & 0xFFFFu)) rest = 1;
                        if (FAST || s + 3 < stages) lds_landed_but<LOADS>();
                        else lds_landed();
                        if (FAST || s + 2 < stages) read_raw(rot2);
                    }
                    fy[(P + 1) & 1][j] = read_y(P ^ 1, 0, j);
#pragma unroll
                    for (int i = j * FD / FN; i < (j + 1) * FD / FN; ++i) fx[P ^ 1][i] = read_x(P ^ 1, i);
                    if (j == 2 && (FAST || s + 2 < stages)) convert_y(fast, 0, s + 2, P);
                    if (FAST || s + 4 < stages) load(fast, j, s + 4, rot1);
                }
#pragma unroll
                for (int i = 0; i < FD; ++i)
                    acc[i][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[P][i], fy[(P + p) & 1][j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);  // keeps the reads where they stand, ahead of their use
            }
        }
    };
    static_assert(LOADS == FN, "a load a step");
    if (stages > 0) {
        if (threadIdx.x == 0) rest = 0;
        load_all(0);
        if (stages > 1) load_all(1);
        if (stages > 2) load_all(2);
        if (stages > 2) lds_landed_but<2 * LOADS>();
        else lds_landed();
        read_raw(0);
#pragma unroll
        for (int i = 0; i < YN; ++i) convert_y(std::false_type{}, i, 0, 0);
#pragma unroll
        for (int h = 0; h < XH; ++h) convert_x(std::false_type{}, h, 0, 0);
        if (stages > 3) {
            load_all(3);
            lds_landed_but<2 * LOADS>();
        } else {
            lds_landed();
        }
        if (stages > 1) {
            read_raw(1);
            convert_y(std::false_type{}, 0, 1, 1);
        }
#pragma unroll
        for (int i = 0; i < FD; ++i) fx[0][i] = read_x(0, i);
#pragma unroll
        for (int j = 0; j < FN; ++j) fy[0][j] = read_y(0, 0, j);
        using std::integral_constant;
        int s = 0, rot = 0;
        auto turn = [&] { rot = rot == 2 ? 0 : rot + 1; };
        for (; s + 6 < stages; s += 2) {
            stage(integral_constant<int, 0>{}, std::true_type{}, s, rot);
            turn();
            stage(integral_constant<int, 1>{}, std::true_type{}, s + 1, rot);
            turn();
        }
#pragma unroll 1
        for (; s < stages; s += 2) {
            stage(integral_constant<int, 0>{}, std::false_type{}, s, rot);
            turn();
            if (s + 1 < stages) stage(integral_constant<int, 1>{}, std::false_type{}, s + 1, rot);
            turn();
        }
        if (__builtin_expect(rest, 0)) {
            const int64_t nw = n0 + wn * FN * 16, dw = d0 + wd * FD * 16;
            const int64_t t_end = t_first + tokens;
            if (rest_matters<FN, FD>(g, acc, nw, dw, t_first, t_end)) add_rest<FN, FD>(g, acc, nw, dw, t_first, t_end);
        }
    }
    store_dw<FN, FD>(g, acc, n0 + wn * FN * 16, d0 + wd * FD * 16);
}

// dW (+)= the splits' partial sums.  A block takes 256 / G pieces of four
// values with G waves each: wave i of them adds splits i, i + G, ..., several
// loads on their way at a time, and the G sums are added in the waves' order.
template <int G>
__global__ void __launch_bounds__(256)
k_ckpt8_wgrad_join(const float* __restrict__ part, int32_t splits, int64_t n, int64_t dim, int64_t ldp,
                   void* __restrict__ out, int64_t ldw, int32_t out_bf16, int32_t accumulate) {
    constexpr int PB = 256 / G;  // pieces of a block
    __shared__ f32x4 sums[G > 1 ? 256 : 1];
    const int64_t pieces_row = ldp / 4, total = n * pieces_row, stride = n * ldp;
    const int at = threadIdx.x % PB, first = threadIdx.x / PB;
    for (int64_t id0 = (int64_t)blockIdx.x * PB; id0 < total; id0 += (int64_t)gridDim.x * PB) {
        const int64_t id = min(id0 + at, total - 1);
        const float* p = part + id * 4;
        f32x4 v{};
        for (int s = first; s < splits; s += 4 * G) {
            f32x4 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = ld_f4(p + (int64_t)min(s + i * G, splits - 1) * stride);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s + i * G < splits) v = s == first && i == 0 ? q[0] : v + q[i];
        }
        if constexpr (G > 1) {
            sums[threadIdx.x] = v;
            __syncthreads();
            if (first == 0) {
#pragma unroll
                for (int i = 1; i < G; ++i) v += sums[i * PB + at];
            }
            __syncthreads();
            if (first != 0) continue;
        }
        if (id0 + at >= total) continue;
        const int64_t r = id / pieces_row, d = (id - r * pieces_row) * 4;
        if (out_bf16) {
            BF16* o = static_cast<BF16*>(out) + r * ldw + d;
            if (d + 4 <= dim) *reinterpret_cast<u32x2_a2*>(o) = u32x2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
            else
                for (int e = 0; e < 4; ++e)
                    if (d + e < dim) put(o + e, v[e]);
            continue;
        }
        float* o = static_cast<float*>(out) + r * ldw + d;
        if (d + 4 <= dim) {
            *reinterpret_cast<f32x4_a4*>(o) = accumulate ? *reinterpret_cast<const f32x4_a4*>(o) + v : v;
        } else {
            for (int e = 0; e < 4; ++e)
                if (d + e < dim) o[e] = accumulate ? o[e] + v[e] : v[e];
        }
    }
}

// ------------------------------------------------------------------ plan
// Tile and number of token splits: the pair whose measured parts add up to
// the least time.  A round is what all 256 compute units do at one time
// (`slots` blocks); it takes `stage_us` for each 32 tokens and `store_us` at
// its end; joining splits takes a launch and the traffic of their sums.
// Measured against each other, whole calls:
// bf16 (tokens x n x dim): 4096 x 4096 x 4096 256 x 256 115 us, 128 x 128 168;
// 2048 x 2048 x 2048 128 x 128 34 us, 256 x 256 58; 4096 x 1024 x 1024 128 x
// 128 in 1 split 56 us, 2 37, 4 27, 16 39; 16384 x 1024 x 1024 256 x 256 in 16
// splits 54 us, 128 x 128 in 8 56.
// fp32: 4096 x 4096 x 4096 128 x 256 347 us, 128 x 128 494; 2048 x 2048 x 2048
// 128 x 256 in 2 splits 64 us, 128 x 128 in 1 68; 4096 x 1024 x 1024 128 x 256
// in 8 splits 40 us, 128 x 128 in 4 47; 1027 x 510 x 770 in 9 splits 128 x 128
// 19.9 us, 128 x 256 21.8.
struct Shape {
    int bn, bd, slots;
    float stage_us, store_us;
    float alone_us;  // stage_us when at most 256 blocks run, one a compute unit
};
constexpr Shape kBf16Shapes[] = {{128, 128, 512, 0.75f, 4.0f, 0.45f}, {256, 256, 256, 0.83f, 8.0f, 0.83f}};
constexpr Shape kF32Shapes[] = {{128, 128, 256, 0.97f, 5.0f, 0.97f}, {128, 256, 256, 1.33f, 8.0f, 1.33f}};

struct Plan {
    int bd;  // input channels of a tile
    int32_t splits;
    int64_t rows_per_split;
};

Plan plan_of(int64_t rows, int64_t n, int64_t dim, bool bf16) {
    Plan best{128, 1, 64};
    double least = 0;
    const int64_t units = rows > 0 ? (rows + 63) / 64 : 1;  // splits are whole pairs of stages
    for (const Shape& shape : bf16 ? kBf16Shapes : kF32Shapes) {
        const int64_t tiles = ((n + shape.bn - 1) / shape.bn) * ((dim + shape.bd - 1) / shape.bd);
        for (const int64_t want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (want > units) break;
            const int64_t per = (units + want - 1) / want, splits = (units + per - 1) / per;
            const int64_t blocks = tiles * splits, rounds = (blocks + shape.slots - 1) / shape.slots;
            const double stage_us = blocks <= 256 ? shape.alone_us : shape.stage_us;
            double us = (double)rounds * (2.0 * (double)per * stage_us + shape.store_us);
            if (splits > 1)
                us += 2.8 + 0.1 * (double)splits + (double)(splits + 1) * (double)n * (double)dim * (4.0 / 8e6);
            if (least == 0 || us < least) {
                least = us;
                best = Plan{shape.bd, (int32_t)splits, per * 64};
            }
        }
    }
    return best;
}

int64_t part_pitch(int64_t dim) { return (dim + 3) & ~int64_t(3); }

template <int BD>
hipError_t launch_pipe_f32(const Args& g, int32_t splits, hipStream_t stream) {
    const dim3 grid((unsigned)(((g.n + 127) / 128) * ((g.dim + BD - 1) / BD)), (unsigned)splits);
    hipLaunchKernelGGL((k_ckpt8_wgrad_pipe_f32<BD>), grid, dim3(512), 0, stream, g);
    return hipGetLastError();
}

template <int BN, int BD, int WN, int WD>
hipError_t launch_pipe(const Args& g, int32_t splits, hipStream_t stream) {
    const dim3 grid((unsigned)(((g.n + BN - 1) / BN) * ((g.dim + BD - 1) / BD)), (unsigned)splits);
    hipLaunchKernelGGL((k_ckpt8_wgrad_pipe<BN, BD, WN, WD>), grid, dim3(WN * WD * WAVE), 0, stream, g);
    return hipGetLastError();
}

template <int P, int B, int WN, int WD, int TK>
hipError_t launch_tile(const Args& g, int32_t splits, hipStream_t stream) {
    const dim3 grid((unsigned)(((g.n + B - 1) / B) * ((g.dim + B - 1) / B)), (unsigned)splits);
    hipLaunchKernelGGL((k_ckpt8_wgrad<P, B, B, WN, WD, TK>), grid, dim3(WN * WD * WAVE), 0, stream, g);
    return hipGetLastError();
}

// g.out, g.ldw: the partial sums of launch_pipe or launch_tile
hipError_t launch_join(const Args& g, int32_t splits, void* dw, bool dw_bf16, int64_t ldw, bool accumulate,
                       hipStream_t stream) {
    const int64_t pieces = g.n * (g.ldw / 4);
    auto run = [&](auto kernel, int per_block) {
        const int64_t blocks = (pieces + per_block - 1) / per_block;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256), 0, stream,
                           static_cast<const float*>(g.out), splits, g.n, g.dim, g.ldw, dw, ldw, (int32_t)dw_bf16,
                           (int32_t)accumulate);
        return hipGetLastError();
    };
    // Four waves a piece where one would leave compute units idle: 64 splits of
    // 128 x 128 5.0 us against 9.9; 9 splits of 510 x 770 9.2 against 8.0.
    return pieces <= 65536 ? run(k_ckpt8_wgrad_join<4>, 64) : run(k_ckpt8_wgrad_join<1>, 256);
}

}  // namespace

int64_t ckpt8_wgrad_workspace(int64_t rows, int64_t n, int64_t dim, bool bf16) {
    const Plan p = plan_of(rows, n, dim, bf16);
    return p.splits > 1 ? p.splits * n * part_pitch(dim) * 4 : 0;
}

hipError_t launch_ckpt8_wgrad(const void* dy, bool dy_bf16, int64_t ldy, const void* codes, const void* exps,
                              int64_t rows, int64_t n, int64_t dim, void* dw, bool dw_bf16, int64_t ldw,
                              bool accumulate, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(rows, n, dim, dy_bf16);
    Args g{};
    g.dy = dy;
    g.ldy = ldy;
    g.codes = static_cast<const uint8_t*>(codes);
    g.exps = static_cast<const uint8_t*>(exps);
    g.pitch = (dim + 31) / 32 * 32;
    g.epitch = (dim + 127) / 128 * 4;
    g.rows = rows;
    g.n = n;
    g.dim = dim;
    g.rows_per_split = p.rows_per_split;
    g.out = p.splits > 1 ? workspace : dw;
    g.ldw = p.splits > 1 ? part_pitch(dim) : ldw;
    g.split_stride = n * part_pitch(dim);
    g.out_bf16 = p.splits > 1 ? 0 : dw_bf16;
    g.accumulate = p.splits > 1 ? 0 : accumulate;
    hipError_t e;
    if (!dy_bf16) {
        if (n < 4) e = launch_tile<3, 128, 2, 2, 64>(g, p.splits, stream);
        else if (p.bd == 256) e = launch_pipe_f32<256>(g, p.splits, stream);
        else e = launch_pipe_f32<128>(g, p.splits, stream);
    } else {
        if (n < 8) e = launch_tile<1, 128, 2, 2, 64>(g, p.splits, stream);
        else if (p.bd == 256) e = launch_pipe<256, 256, 2, 4>(g, p.splits, stream);
        else e = launch_pipe<128, 128, 2, 2>(g, p.splits, stream);
    }
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_join(g, p.splits, dw, dw_bf16, ldw, accumulate, stream);
}

}  // namespace qc
