// k_adamw.hip -- the optimizer's side of a tensor list: the norm of the
// gradients, and one AdamW step over parameters and gradients read in place,
// its states fp32 arrays or 8-bit codes laid out for the concatenation.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - rate * m / (sqrt(v) * root + eps)
//
// with rate = lr / (1 - b1^t) and root = 1 / sqrt(1 - b2^t).
//
// Bound by HBM where n is large: the norm reads g once, the step g, p, m and v
// and writes the last three (268 M elements: norm of fp32 170 us, 6.3 TB/s, as
// part of it still lies in the last cache; the step in fp32 1300 to 1430 us, 5.3
// to 5.8 TB/s; bf16 parameters and gradients with fp32 states 1000 us, 5.9, and
// with master weights 1330, 5.7; with 8-bit states 645 to 675 us, 4.0 to 4.2, and
// 780 to 855, 5.0 to 5.5; states encoded 213 us, 6.3, decoded to fp32 212 to 220,
// to bf16 131 to 141).
// Short lists are bound by loads that wait for each other.
#include "qc_matrix.hpp"
#include "qc_launch.hpp"

#include "qc.h"

namespace qc {
namespace {

// --------------------------------------------------------- tensor lists
// A block of 256 threads takes a run of passes of 2048 elements.  It keeps the
// tensor that it is in, so a pass inside one tensor loads no table (with the
// index looked up for each segment of 4096, three loads before the first value,
// the norm of 268 M bf16 gradients took 274 us).  Where a pass may reach into
// another tensor each lane searches the few of its segment for its fours, and
// where a four lies in more than one, for each element.
//
// 32 lanes hold 256 elements, a block of the 8-bit states; a lane four in each
// half of them, so that an access of fp32 covers 512 bytes without gaps.
constexpr int kThreads = 256, kPass = kThreads * 8, kFour = 4;
constexpr int kMaxRuns = 2048;  // blocks of the norm: eight for each compute unit

__device__ __forceinline__ int lane_first() { return (threadIdx.x >> 5) * 256 + (threadIdx.x & 31) * kFour; }
constexpr int kHalf = 128;  // from a lane's first four to its second

typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// Four neighbouring values, `left` of which exist (the rest read as +0).
__device__ __forceinline__ void load4(const float* p, int left, float (&v)[4]) {
    if (left >= 4) {
        const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void load4(const BF16* p, int left, float (&v)[4]) {
    if (left >= 4) {
        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a2*>(p));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void store4(float* p, int left, const float (&v)[4]) {
    if (left >= 4) {
        const u32x4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = v[i];
    }
}
__device__ __forceinline__ void store4(BF16* p, int left, const float (&v)[4]) {
    if (left >= 4) {
        const u32x2 w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2_a2*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) put(p + i, v[i]);
    }
}

struct Tables {
    const int64_t* off;
    const int32_t* seg;
    int32_t T;
    int64_t n;
    int64_t passes_per_run;
};

// The tensors that the pass from element i0 may reach into (a pass lies in one
// segment).  Index values are clamped, so that a corrupt index cannot send an
// access outside the tables.
struct Range {
    int32_t lo, hi;
};
__device__ __forceinline__ int32_t clamped(int32_t t, int32_t lo, int32_t hi) { return min(max(t, lo), hi); }
__device__ __forceinline__ Range range_at(const Tables& l, int64_t i0) {
    const int32_t* seg = l.seg + (i0 >> QC_INDEX_SHIFT);
    const int32_t first = seg[0], next = seg[1], lo = clamped(first, 0, l.T - 1);
    return Range{lo, clamped(next, lo, l.T - 1)};
}

// A tensor begins and ends at these elements of the pass (those before and
// behind it made one), and element 0 of the pass would lie at `param`, `grad`.
__device__ __forceinline__ int32_t in_pass(const Tables& l, int64_t i0, int64_t off) {
    return (int32_t)max(min(min(off, l.n) - i0, (int64_t)kPass), (int64_t)-1);
}
template <class T>
__device__ __forceinline__ T* from_pass(T* p, int64_t i0, int64_t off) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(i0 - off) * sizeof(T));
}

// Up to kNear of the range's tensors at a time, read side by side, a thread a
// tensor, so that the searches wait for LDS and not for one load from memory
// after the other (24 tensors of 40,000 elements in all: the step 9.5 us with
// searches in memory, 7.3 here, the norm 5.6 and 4.7; 77 of 3,000,000, bf16 and
// 8-bit states: 19.4 and 17.6 us, the norm 9.5 and 6.8).
constexpr int kNear = kThreads - 1;
template <class P, class G>
struct Near {
    int32_t begins[kNear + 1];
    P* params[kNear];
    G* grads[kNear];
};
template <class P, class G>
struct Part {
    const Near<P, G>& near;
    int32_t lo, hi;
    __device__ __forceinline__ int32_t begin(int32_t t) const { return near.begins[t - lo]; }
    __device__ __forceinline__ P* param(int32_t t) const { return near.params[t - lo]; }
    __device__ __forceinline__ G* grad(int32_t t) const { return near.grads[t - lo]; }
};
// f(part) for each part of the range; every thread of the block calls this.
// `filled`: the last call was for the same pass, and there is one part.
template <class P, class G, class F>
__device__ __forceinline__ void for_parts(Near<P, G>& near, const Tables& l, int64_t i0, const Range& r, P* const* ps,
                                          G* const* gs, bool filled, F f) {
    for (int32_t lo = r.lo;; lo += kNear) {
        const int32_t i = threadIdx.x, count = min(r.hi - lo + 1, kNear);
        if (!filled) {
            int64_t off = 0;
            P* p = nullptr;
            G* g = nullptr;
            if (i <= count) off = l.off[lo + i];
            if (i < count) {
                if (ps) p = ps[lo + i];
                g = gs[lo + i];
            }
            __syncthreads();  // of the part before no thread reads any more
            if (i <= count) near.begins[i] = in_pass(l, i0, off);
            if (i < count) {
                near.params[i] = from_pass(p, i0, off);
                near.grads[i] = from_pass(g, i0, off);
            }
            __syncthreads();
        }
        f(Part<P, G>{near, lo, lo + count - 1});
        if (r.hi - lo < kNear) break;
    }
}

// The tensors of N elements, e(j) the place of element j in the pass: of those
// of the part, the last that begins at the element or before it, else the first.
// The searches go on side by side.
template <int N, class L, class E>
__device__ __forceinline__ void tensors_of(const L& l, E e, int32_t (&t)[N]) {
    int32_t last[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        t[j] = l.lo;
        last[j] = l.hi;
    }
    // every one halves the same range, first to last, so they end together
    for (int32_t span = l.hi - l.lo; span > 0; span >>= 1) {
        int32_t mid[N], v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            mid[j] = (t[j] + last[j] + 1) >> 1;
            v[j] = l.begin(mid[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (v[j] <= e(j)) t[j] = mid[j];
            else last[j] = mid[j] - 1;
        }
    }
}

// A lane's two fours, from e and e + half: each in one tensor, or over several.
struct Fours {
    int32_t t[2];
    bool whole[2];
};
template <class L>
__device__ __forceinline__ Fours fours_of(const L& l, int e, int half) {
    Fours f;
    tensors_of<2>(l, [&](int q) { return e + q * half; }, f.t);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int first = e + q * half;
        f.whole[q] = l.begin(f.t[q]) <= first && first + kFour <= l.begin(f.t[q] + 1);
    }
    return f;
}

// Four elements that lie over several tensors.  Those of another part, past the
// end, or of tables that contradict each other are not there.
struct Places {
    int32_t t[kFour];
    bool there[kFour];
};
template <class L>
__device__ __forceinline__ Places places_of(const L& l, int e) {
    Places s;
    tensors_of<kFour>(l, [&](int j) { return e + j; }, s.t);
#pragma unroll
    for (int j = 0; j < kFour; ++j) s.there[j] = l.begin(s.t[j]) <= e + j && e + j < l.begin(s.t[j] + 1);
    return s;
}
// p(t): where element 0 of the pass would lie in tensor t
template <class F>
__device__ __forceinline__ void load_places(F p, const Places& s, int e, float (&v)[kFour]) {
#pragma unroll
    for (int j = 0; j < kFour; ++j) {
        const auto at = p(s.t[j]);
        if (s.there[j]) v[j] = to_f32(at[e + j]);
    }
}
template <class F>
__device__ __forceinline__ void store_places(F p, const Places& s, int e, const float (&v)[kFour]) {
#pragma unroll
    for (int j = 0; j < kFour; ++j) {
        const auto at = p(s.t[j]);
        if (s.there[j]) put(at + e + j, v[j]);
    }
}

// The tensor that the last pass of a block lay in entirely.
struct Cursor {
    int32_t t;
    int64_t from, to;
    __device__ __forceinline__ bool holds(int64_t i0, int64_t end) const { return i0 >= from && end <= to; }
};

// ------------------------------------------------------------ 8-bit states
// A code is the top bits of the fp32 number y = |x| / scale, whose exponent
// field counts from 2^-15 on: LOW bits of the fraction are rounded away, up
// where they are above 2^LOW (1 - u).
template <int KIND>
struct State {
    static constexpr bool SIGNED = KIND == QC_STATE_M;
    static constexpr int LOW = SIGNED ? 20 : 19, TOP = SIGNED ? 127 : 255;
    static constexpr uint32_t FIRST = SIGNED ? 896 : 1792;
    static constexpr uint32_t SHIFT = SIGNED ? 0u : 0x80000000u;  // of u32
};

// 2^32 / rho^2 and 2^32 / rho, rho = 1.3247... the real root of x^3 = x + 1 (the
// plastic number): the additive recurrence of two dimensions with even gaps
// that Martin Roberts published as R2, elements along one and steps along the
// other.
constexpr uint32_t kDitherElem = 0x91E10DA5u, kDitherStep = 0xC13FA9A9u;

template <int KIND>
__device__ __forceinline__ float state_value(uint32_t code) {
    using S = State<KIND>;
    const uint32_t mag = S::SIGNED ? code & 127u : code;
    const float f = mag ? __uint_as_float((S::FIRST + mag) << S::LOW) : 0.0f;
    return S::SIGNED ? __uint_as_float(__float_as_uint(f) | ((code & 128u) << 24)) : f;
}

// Scale and reciprocal of a block whose largest magnitude has these bits.
template <int KIND>
__device__ __forceinline__ float state_scale(uint32_t amax_bits, float& inv) {
    using S = State<KIND>;
    const float rest = 1.0f / __builtin_bit_cast(float, (S::FIRST + S::TOP) << S::LOW);
    const float s = fmaxf(__uint_as_float(amax_bits) * rest, 0x1p-100f);
    const bool zero = amax_bits == 0, nan = amax_bits >= kInfBits;
    inv = zero || nan ? 0.0f : 1.0f / s;
    return nan ? __uint_as_float(0x7FC00000u) : (zero ? 0.0f : s);
}

// u: the 32 bits of the threshold.  inv == 0: code 0 (of NaNs too, as no
// comparison holds).  Below the first code's value y + the threshold comes to
// that code at most, and m becomes 0 where y is not above u of that value.
template <int KIND>
__device__ __forceinline__ uint32_t state_code(float x, float inv, uint32_t u) {
    using S = State<KIND>;
    constexpr float kLeast = __builtin_bit_cast(float, (S::FIRST + 1) << S::LOW);
    const float y = fabsf(x) * inv;
    const int32_t up = (int32_t)(__float_as_uint(y) + (u >> (32 - S::LOW)) - (S::FIRST << S::LOW)) >> S::LOW;
    uint32_t c = (uint32_t)min(max(up, 1), S::TOP);
    if (S::SIGNED) c |= (__float_as_uint(x) >> 24) & 128u;
    return y > (S::SIGNED ? (float)(u >> 8) * (kLeast * 0x1p-24f) : 0.0f) ? c : 0u;
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int left) {
    if (left >= 4) return ld_stream_u32(p);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) w |= (uint32_t)p[i] << (8 * i);
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int left, uint32_t w) {
    if (left >= 4) {
        st_u32(p, w);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = (uint8_t)(w >> (8 * i));
    }
}

template <int KIND>
__device__ __forceinline__ void state_values(uint32_t codes, float scale, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = state_value<KIND>((codes >> (8 * i)) & 255u) * scale;
}

// Codes of a lane's two fours, `u` the threshold of the first; 32 neighbouring
// lanes hold a block, all of them call this.
template <int KIND>
__device__ __forceinline__ float state_codes(const float (&x)[2][4], uint32_t u, uint32_t each, uint32_t (&w)[2]) {
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = umax(amax, abs_bits(x[q][i]));
    amax = group_max_u32<32>(amax);
    float inv;
    const float scale = state_scale<KIND>(amax, inv);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        w[q] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[q] |= state_code<KIND>(x[q][i], inv, u + State<KIND>::SHIFT + (uint32_t)(q * kHalf + i) * each) << (8 * i);
    }
    return scale;
}

// Flat arrays of n elements, laid out over lanes as above; every lane of a wave
// runs the same passes.
template <int KIND>
__global__ void __launch_bounds__(kThreads)
k_enc_state8(const float* __restrict__ x, int64_t n, uint8_t* __restrict__ codes, float* __restrict__ scale) {
    for (int64_t first = (int64_t)blockIdx.x * kPass; first < n; first += (int64_t)gridDim.x * kPass) {
        const int e = lane_first(), left = (int)min(n - first, (int64_t)kPass) - e;
        float v[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) load4(x + first + e + q * kHalf, left - q * kHalf, v[q]);
        uint32_t w[2];
        const float s = state_codes<KIND>(v, 0x80000000u - State<KIND>::SHIFT, 0u, w);
#pragma unroll
        for (int q = 0; q < 2; ++q) store_codes(codes + first + e + q * kHalf, left - q * kHalf, w[q]);
        if (left > 0 && (threadIdx.x & 31) == 0) scale[first / QC_STATE_BLOCK + threadIdx.x / 32] = s;
    }
}

template <int KIND, class T>
__global__ void __launch_bounds__(kThreads)
k_dec_state8(const uint8_t* __restrict__ codes, const float* __restrict__ scale, int64_t n, T* __restrict__ out) {
    for (int64_t first = (int64_t)blockIdx.x * kPass; first < n; first += (int64_t)gridDim.x * kPass) {
        const int e = lane_first(), left = (int)min(n - first, (int64_t)kPass) - e;
        const float s = left > 0 ? scale[first / QC_STATE_BLOCK + threadIdx.x / 32] : 0.0f;
        uint32_t w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) w[q] = load_codes(codes + first + e + q * kHalf, left - q * kHalf);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[4];
            state_values<KIND>(w[q], s, v);
            store4(out + first + e + q * kHalf, left - q * kHalf, v);
        }
    }
}

// ------------------------------------------------------------------ AdamW

struct Wide {  // fp32 states
    float* m;
    float* v;
};
struct Narrow {
    uint8_t* mc;
    float* ms;
    uint8_t* rc;
    float* rs;
};

struct Rates {
    float decay, rate, root, scale;
    uint32_t t;
};

// What the step's constants are: the host's, or from the device's {lr, t}.
__device__ __forceinline__ Rates rates_of(const AdamwStep& s) {
    Rates r{s.decay, s.rate, s.root, s.grad_scale ? *s.grad_scale : 1.0f, s.t};
    if (s.schedule) {
        const double lr = s.schedule[0], t = s.schedule[1];
        r.decay = (float)(1.0 - lr * s.weight_decay);
        r.rate = (float)(lr / (1.0 - exp2(t * s.log2_beta1)));
        r.root = (float)(1.0 / sqrt(1.0 - exp2(t * s.log2_beta2)));
        r.t = (uint32_t)(int64_t)t;
    }
    return r;
}

// Five blocks a compute unit where the registers are enough (3 M elements, 8-bit
// states: 17.2 us, with four 17.8); with master weights they would spill.
template <class P, class G, class S, bool MASTER>
__global__ void __launch_bounds__(kThreads, MASTER ? 4 : 5)
k_adamw(Tables l, P* const* __restrict__ params, G* const* __restrict__ grads, float* __restrict__ master, S st,
        AdamwStep step) {
    constexpr bool WIDE = std::is_same<S, Wide>::value;
    const Rates k = rates_of(step);
    const int64_t first = (int64_t)blockIdx.x * l.passes_per_run * kPass;
    const int64_t end = min(first + l.passes_per_run * kPass, l.n);
    __shared__ Near<P, G> near;
    const int e = lane_first();
    Cursor cur{0, 0, 0};
#pragma unroll 1
    for (int64_t i0 = first; i0 < end; i0 += kPass) {
        const int left = (int)min(l.n - i0, (int64_t)kPass) - e;
        // the states' places need no table: their loads go first
        float m[2][4], v[2][4], p[2][4], g[2][4];
        uint32_t mc[2], rc[2];
        float ms = 0.0f, rs = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int at = e + q * kHalf, some = left - q * kHalf;
            if constexpr (WIDE) {
                load4(st.m + i0 + at, some, m[q]);
                load4(st.v + i0 + at, some, v[q]);
            } else {
                mc[q] = load_codes(st.mc + i0 + at, some);
                rc[q] = load_codes(st.rc + i0 + at, some);
            }
            if (MASTER) load4(master + i0 + at, some, p[q]);
        }
        const int64_t block = i0 / QC_STATE_BLOCK + threadIdx.x / 32;
        if constexpr (!WIDE) {
            if (left > 0) {
                ms = st.ms[block];
                rs = st.rs[block];
            }
        }
        Range range{0, 0};
        if (!cur.holds(i0, i0 + kPass)) {
            range = range_at(l, i0);
            if (range.lo == range.hi) cur = Cursor{range.lo, l.off[range.lo], min(l.off[range.lo + 1], l.n)};
        }
        const bool one = cur.holds(i0, i0 + kPass);
        bool whole[2] = {one, one};
        P* pq[2];
        if (one) {
            pq[0] = pq[1] = from_pass(params[cur.t], i0, cur.from);
            const G* gp = from_pass(grads[cur.t], i0, cur.from);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                load4(gp + e + q * kHalf, kFour, g[q]);
                if (!MASTER) load4(const_cast<const P*>(pq[q]) + e + q * kHalf, kFour, p[q]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < kFour; ++j) {
                    g[q][j] = 0.0f;
                    if (!MASTER) p[q][j] = 0.0f;
                }
            for_parts(near, l, i0, range, params, grads, false, [&](const auto& from) {
                const Fours f = fours_of(from, e, kHalf);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = e + q * kHalf;
                    if (f.whole[q]) {
                        whole[q] = true;
                        pq[q] = from.param(f.t[q]);
                        load4(const_cast<const G*>(from.grad(f.t[q])) + at, kFour, g[q]);
                        if (!MASTER) load4(const_cast<const P*>(pq[q]) + at, kFour, p[q]);
                    }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = e + q * kHalf;
                    if (!whole[q]) {
                        const Places s = places_of(from, at);
                        load_places([&](int t) { return from.grad(t); }, s, at, g[q]);
                        if (!MASTER) load_places([&](int t) { return from.param(t); }, s, at, p[q]);
                    }
                }
            });
        }
        float r[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if constexpr (!WIDE) {
                state_values<QC_STATE_M>(mc[q], ms, m[q]);
                state_values<QC_STATE_R>(rc[q], rs, v[q]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = g[q][e] * k.scale, old = WIDE ? v[q][e] : v[q][e] * v[q][e];
                // no fused multiply-add: the states' bits are those of the formula as it is
                // written, or a code that hangs on the last bit would differ from the host's
                m[q][e] = m[q][e] * step.beta1 + x * step.rest1;
                v[q][e] = old * step.beta2 + x * x * step.rest2;
                r[q][e] = sqrtf(v[q][e]);
                const float den = __builtin_fmaf(r[q][e], k.root, step.eps);
                // the hardware's reciprocal is off by an ulp; den is 0 or a normal number
                p[q][e] = p[q][e] * k.decay - k.rate * m[q][e] * __builtin_amdgcn_rcpf(den);
            }
        }
        if constexpr (!WIDE) {
            // every lane of the wave takes part; those past the end hold zeros
            const uint32_t u = ((uint32_t)i0 + e) * kDitherElem + k.t * kDitherStep;
            ms = state_codes<QC_STATE_M>(m, u, kDitherElem, mc);
            rs = state_codes<QC_STATE_R>(r, u, kDitherElem, rc);
            if (left > 0 && (threadIdx.x & 31) == 0) {
                st.ms[block] = ms;
                st.rs[block] = rs;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int at = e + q * kHalf, some = left - q * kHalf;
            if constexpr (WIDE) {
                store4(st.m + i0 + at, some, m[q]);
                store4(st.v + i0 + at, some, v[q]);
            } else {
                store_codes(st.mc + i0 + at, some, mc[q]);
                store_codes(st.rc + i0 + at, some, rc[q]);
            }
            if (MASTER) store4(master + i0 + at, some, p[q]);
            if (whole[q]) store4(pq[q] + at, kFour, p[q]);
        }
        if (!one) {
            for_parts(near, l, i0, range, params, grads, range.hi - range.lo < kNear, [&](const auto& to) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = e + q * kHalf;
                    if (!whole[q]) store_places([&](int t) { return to.param(t); }, places_of(to, at), at, p[q]);
                }
            });
        }
    }
}

// ------------------------------------------------------------------- norm
// Squares are summed in 64 bits, so none overflows or vanishes.  Each block
// leaves the sum of its run; a second kernel adds those up, always in the same
// order.  Inside a tensor a thread has the loads of four passes on their way.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if (lane_id() == 0) lds[wave_id()] = v;
    __syncthreads();
    double sum = lds[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += lds[w];
    return sum;
}

__device__ __forceinline__ double add_squares(double sum, const float (&g)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = __builtin_fma((double)g[e], (double)g[e], sum);
    return sum;
}

template <class G>
__global__ void __launch_bounds__(kThreads)
k_norm_parts(Tables l, G* const* __restrict__ grads, double* __restrict__ parts) {
    __shared__ double lds[4];
    constexpr int U = 8;  // fours: of four passes
    const int64_t first = (int64_t)blockIdx.x * l.passes_per_run * kPass;
    const int64_t end = min(first + l.passes_per_run * kPass, l.n);
    __shared__ Near<const G, G> near;
    const int e = threadIdx.x * kFour;
    Cursor cur{0, 0, 0};
    double sum = 0.0;
#pragma unroll 1
    for (int64_t i0 = first; i0 < end;) {
        Range range{0, 0};
        if (!cur.holds(i0, i0 + kPass)) {
            range = range_at(l, i0);
            if (range.lo == range.hi) cur = Cursor{range.lo, l.off[range.lo], min(l.off[range.lo + 1], l.n)};
        }
        const bool one = cur.holds(i0, i0 + kPass);
        const G* gp = one ? from_pass(grads[cur.t], i0, cur.from) : nullptr;
        if (one && cur.holds(i0, i0 + U / 2 * kPass) && i0 + U / 2 * kPass <= end) {
            float g[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) load4(gp + e + u * (kPass / 2), kFour, g[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) sum = add_squares(sum, g[u]);
            i0 += U / 2 * kPass;
            continue;
        }
        float g[2][4];
        if (one) {
#pragma unroll
            for (int q = 0; q < 2; ++q) load4(gp + e + q * (kPass / 2), kFour, g[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < kFour; ++j) g[q][j] = 0.0f;
            for_parts(near, l, i0, range, static_cast<const G* const*>(nullptr), grads, false, [&](const auto& from) {
                const Fours f = fours_of(from, e, kPass / 2);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (f.whole[q])
                        load4(const_cast<const G*>(from.grad(f.t[q])) + e + q * (kPass / 2), kFour, g[q]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int at = e + q * (kPass / 2);
                    if (!f.whole[q]) load_places([&](int t) { return from.grad(t); }, places_of(from, at), at, g[q]);
                }
            });
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) sum = add_squares(sum, g[q]);
        i0 += kPass;
    }
    sum = block_sum<kThreads / WAVE>(sum, lds);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// Two loads a thread for all parts there can be, side by side (1465 parts 2.2 us,
// with 256 threads and a loop 3.0; 20 parts 2.0 and 1.7).
constexpr int kJoin = kMaxRuns / 2;
__global__ void __launch_bounds__(kJoin)
k_norm_join(const double* __restrict__ parts, int blocks, double max_norm, float* __restrict__ out) {
    __shared__ double lds[kJoin / WAVE];
    double v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = threadIdx.x + i * kJoin < blocks ? parts[threadIdx.x + i * kJoin] : 0.0;
    const double sum = block_sum<kJoin / WAVE>(v[0] + v[1], lds);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum), c = max_norm / norm;
        out[0] = (float)norm;
        // an infinite norm clips with a NaN, not with zero, so that it is seen
        out[1] = norm - norm == 0.0 ? (float)(c < 1.0 ? c : 1.0) : __uint_as_float(0x7FC00000u);
    }
}

// Runs of equal length, at most kMaxRuns.
struct Runs {
    int64_t passes;
    int blocks;
};
Runs runs_of(int64_t n, int64_t most) {
    const int64_t all = (n + kPass - 1) / kPass, each = (all + most - 1) / most;
    return Runs{each, (int)((all + each - 1) / each)};
}
Runs norm_runs(int64_t n) { return runs_of(n, kMaxRuns); }
// One pass a block, as far as a grid goes: all blocks at work then read and
// write a few places that move on together (268 M elements, fp32 states, with 1,
// 2 and 4 passes 1430, 1445 and 1520 us; 8-bit 845, 840, 860; 3 M elements, 8-bit,
// 17.1, 21.0, 29.7).
Runs step_runs(int64_t n) { return runs_of(n, kMaxBlocks); }

unsigned grid_of(int64_t n, int64_t each) {
    const int64_t g = (n + each - 1) / each;
    return (unsigned)(g < kMaxBlocks ? g : kMaxBlocks);
}

Tables tables_of(const ListSrc& l, const Runs& r) { return Tables{l.offsets, l.seg_first, l.ntensors, l.n, r.passes}; }

template <class P, class G, class S, bool MASTER>
hipError_t launch_step(const AdamwList& l, const S& st, const AdamwStep& s, hipStream_t stream) {
    const Runs r = step_runs(l.grads.n);
    hipLaunchKernelGGL((k_adamw<P, G, S, MASTER>), dim3(r.blocks), dim3(kThreads), 0, stream, tables_of(l.grads, r),
                       reinterpret_cast<P* const*>(l.params),
                       reinterpret_cast<G* const*>(const_cast<void* const*>(
                           reinterpret_cast<const void* const*>(l.grads.xs))),
                       l.master, st, s);
    return hipGetLastError();
}

template <class G, class S>
hipError_t launch_params(const AdamwList& l, const S& st, const AdamwStep& s, hipStream_t stream) {
    if (!l.p_bf16) return launch_step<float, G, S, false>(l, st, s, stream);
    return l.master ? launch_step<BF16, G, S, true>(l, st, s, stream) : launch_step<BF16, G, S, false>(l, st, s, stream);
}

template <class S>
hipError_t launch_any(const AdamwList& l, const S& st, const AdamwStep& s, hipStream_t stream) {
    return l.g_bf16 ? launch_params<BF16>(l, st, s, stream) : launch_params<float>(l, st, s, stream);
}

}  // namespace

hipError_t launch_adamw(const AdamwList& l, float* m, float* v, const AdamwStep& s, hipStream_t stream) {
    return launch_any(l, Wide{m, v}, s, stream);
}

hipError_t launch_adamw8(const AdamwList& l, uint8_t* m_codes, float* m_scale, uint8_t* r_codes, float* r_scale,
                         const AdamwStep& s, hipStream_t stream) {
    return launch_any(l, Narrow{m_codes, m_scale, r_codes, r_scale}, s, stream);
}

hipError_t launch_encode_state8(int32_t kind, const float* x, int64_t n, uint8_t* codes, float* scale,
                                hipStream_t stream) {
    const dim3 grid(grid_of(n, kPass)), block(kThreads);
    if (kind == QC_STATE_M)
        hipLaunchKernelGGL(k_enc_state8<QC_STATE_M>, grid, block, 0, stream, x, n, codes, scale);
    else
        hipLaunchKernelGGL(k_enc_state8<QC_STATE_R>, grid, block, 0, stream, x, n, codes, scale);
    return hipGetLastError();
}

namespace {

template <int KIND, class T>
hipError_t launch_dec(const uint8_t* codes, const float* scale, int64_t n, T* out, hipStream_t stream) {
    hipLaunchKernelGGL((k_dec_state8<KIND, T>), dim3(grid_of(n, kPass)), dim3(kThreads), 0, stream, codes, scale, n,
                       out);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_dec_as(const uint8_t* codes, const float* scale, int64_t n, void* out, bool bf16,
                         hipStream_t stream) {
    return bf16 ? launch_dec<KIND>(codes, scale, n, static_cast<BF16*>(out), stream)
                : launch_dec<KIND>(codes, scale, n, static_cast<float*>(out), stream);
}

}  // namespace

hipError_t launch_decode_state8(int32_t kind, const uint8_t* codes, const float* scale, int64_t n, void* out,
                                bool bf16, hipStream_t stream) {
    return kind == QC_STATE_M ? launch_dec_as<QC_STATE_M>(codes, scale, n, out, bf16, stream)
                              : launch_dec_as<QC_STATE_R>(codes, scale, n, out, bf16, stream);
}

int64_t grad_norm_workspace(int64_t n) { return n > 0 ? 8 * (int64_t)norm_runs(n).blocks : 0; }

hipError_t launch_grad_norm(const ListSrc& l, bool bf16, double max_norm, void* workspace, float* out,
                            hipStream_t stream) {
    const Runs r = norm_runs(l.n);
    const int blocks = r.blocks;
    double* parts = static_cast<double*>(workspace);
    auto xs = const_cast<void* const*>(reinterpret_cast<const void* const*>(l.xs));
    if (bf16)
        hipLaunchKernelGGL(k_norm_parts<BF16>, dim3(blocks), dim3(kThreads), 0, stream, tables_of(l, r),
                           reinterpret_cast<BF16* const*>(xs), parts);
    else
        hipLaunchKernelGGL(k_norm_parts<float>, dim3(blocks), dim3(kThreads), 0, stream, tables_of(l, r),
                           reinterpret_cast<float* const*>(xs), parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_norm_join, dim3(1), dim3(kJoin), 0, stream, parts, blocks, max_norm, out);
    return hipGetLastError();
}

}  // namespace qc
