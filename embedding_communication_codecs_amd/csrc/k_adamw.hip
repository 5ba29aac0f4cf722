// k_adamw.hip -- the optimizer's side of a tensor list: the norm of the
// gradients, and one AdamW step over parameters and gradients read in place,
// its states fp32 arrays or 8-bit codes laid out for the concatenation.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - rate * m / (sqrt(v) * root + eps)
//
// with rate = lr / (1 - b1^t) and root = 1 / sqrt(1 - b2^t).
#include "qc_matrix.hpp"
#include "qc_launch.hpp"

#include "qc.h"

namespace qc {
namespace {

// --------------------------------------------------------- tensor lists
// A block of 256 threads works on one segment of 2^QC_INDEX_SHIFT = 4096
// elements at a time, so that the index names the tensors of the whole
// segment with two loads.  Where that is one tensor, the address is the
// block's; elsewhere each lane searches the few tensors between, and eight
// elements that lie in more than one are taken one by one.
constexpr int kSeg = 1 << QC_INDEX_SHIFT;
constexpr int kThreads = 256, kEach = 8, kPass = kThreads * kEach, kPasses = kSeg / kPass;

struct Tables {
    const int64_t* off;
    const int32_t* seg;
    int32_t T;
    int64_t n;
};

// The tensors of segment j, first and last; index values are clamped, so that
// a corrupt index cannot send an access outside the tables.
__device__ __forceinline__ void tensors_of(const Tables& l, int64_t j, int32_t& lo, int32_t& hi) {
    const int32_t a = l.seg[j], b = l.seg[j + 1];
    lo = __builtin_amdgcn_readfirstlane(min(max(a, 0), l.T - 1));
    hi = __builtin_amdgcn_readfirstlane(min(max(b, lo), l.T - 1));
}

// Where eight elements from i of the concatenation lie.
struct Span {
    int32_t t;     // the tensor of the first
    int64_t at;    // its index there
    bool whole;    // all eight are in tensor t
};

__device__ __forceinline__ Span span_of(const Tables& l, int32_t lo, int32_t hi, int64_t i) {
    int32_t a = lo, b = hi;
    while (a < b) {
        const int32_t mid = (a + b + 1) >> 1;
        if (l.off[mid] <= i) a = mid;
        else b = mid - 1;
    }
    const int64_t o = l.off[a];
    return Span{a, i - o, i >= o && i + kEach <= min(l.off[a + 1], l.n)};
}

// Calls f(j, tensor, index) for those of the eight elements from i that exist.
template <class F>
__device__ __forceinline__ void each_of(const Tables& l, int32_t t, int32_t hi, int64_t i, F f) {
#pragma unroll 1
    for (int j = 0; j < kEach; ++j) {
        const int64_t g = i + j;
        if (g >= l.n) break;
        while (t < hi && g >= l.off[t + 1]) ++t;
        const int64_t o = l.off[t];
        if (g >= o && g < l.off[t + 1]) f(j, t, g - o);
    }
}

template <class T>
__device__ __forceinline__ void load_span(const Tables& l, T* const* xs, const Span& s, int32_t hi, int64_t i,
                                          float (&v)[kEach]) {
    if (s.whole) {
        load8(const_cast<const T*>(xs[s.t]) + s.at, kEach, v);
    } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j] = 0.0f;
        each_of(l, s.t, hi, i, [&](int j, int32_t t, int64_t at) {
            const float x = to_f32(const_cast<const T*>(xs[t])[at]);
#pragma unroll
            for (int q = 0; q < kEach; ++q) v[q] = q == j ? x : v[q];
        });
    }
}

template <class T>
__device__ __forceinline__ void store_span(const Tables& l, T* const* xs, const Span& s, int32_t hi, int64_t i,
                                           const float (&v)[kEach]) {
    if (s.whole) {
        store8(xs[s.t] + s.at, kEach, v);
    } else {
        each_of(l, s.t, hi, i, [&](int j, int32_t t, int64_t at) {
            float x = 0.0f;
#pragma unroll
            for (int q = 0; q < kEach; ++q) x = q == j ? v[q] : x;
            put(xs[t] + at, x);
        });
    }
}

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

// u: the 32 bits of the threshold.  inv == 0: code 0.
template <int KIND>
__device__ __forceinline__ uint32_t state_code(float x, float inv, uint32_t u) {
    using S = State<KIND>;
    constexpr float kLeast = __builtin_bit_cast(float, (S::FIRST + 1) << S::LOW);
    const float y = fabsf(x) * inv;
    const uint32_t up = (__float_as_uint(y) + (u >> (32 - S::LOW))) >> S::LOW;
    const bool low = S::SIGNED ? y > (float)(u >> 8) * (kLeast * 0x1p-24f) : y > 0.0f;
    uint32_t c = y < kLeast ? (low ? 1u : 0u) : min(up - S::FIRST, (uint32_t)S::TOP);
    if (!(inv > 0.0f)) c = 0u;
    if (S::SIGNED && x < 0.0f && c) c |= 128u;
    return c;
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t left) {
    if (left >= 8) return ld_stream_u2(p);
    u32x2 w = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left, u32x2 w) {
    if (left >= 8) {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

template <int KIND>
__device__ __forceinline__ void state_values(u32x2 codes, float scale, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = state_value<KIND>((codes[i >> 2] >> (8 * (i & 3))) & 255u) * scale;
}

// Codes of eight values; 32 neighbouring lanes hold a block, all of them call this.
template <int KIND>
__device__ __forceinline__ u32x2 state_codes(const float (&x)[8], uint32_t u, uint32_t each, float& scale) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = umax(amax, abs_bits(x[i]));
    amax = group_max_u32<32>(amax);
    float inv;
    scale = state_scale<KIND>(amax, inv);
    u32x2 w = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i >> 2] |= state_code<KIND>(x[i], inv, u + State<KIND>::SHIFT + (uint32_t)i * each) << (8 * (i & 3));
    return w;
}

// Kernels over n elements of flat arrays, eight a thread: blocks of 256
// elements are half waves, and every lane of a wave runs the same passes.
template <int KIND>
__global__ void __launch_bounds__(kThreads)
k_enc_state8(const float* __restrict__ x, int64_t n, uint8_t* __restrict__ codes, float* __restrict__ scale) {
    for (int64_t first = (int64_t)blockIdx.x * kPass; first < n; first += (int64_t)gridDim.x * kPass) {
        const int64_t i = first + threadIdx.x * kEach;
        float v[8], s;
        load8(x + i, n - i, v);
        const u32x2 w = state_codes<KIND>(v, 0x80000000u - State<KIND>::SHIFT, 0u, s);
        if (i < n) {
            store_codes(codes + i, n - i, w);
            if ((threadIdx.x & 31) == 0) scale[i / QC_STATE_BLOCK] = s;
        }
    }
}

template <int KIND, class T>
__global__ void __launch_bounds__(kThreads)
k_dec_state8(const uint8_t* __restrict__ codes, const float* __restrict__ scale, int64_t n, T* __restrict__ out) {
    for (int64_t first = (int64_t)blockIdx.x * kPass; first < n; first += (int64_t)gridDim.x * kPass) {
        const int64_t i = first + threadIdx.x * kEach;
        if (i < n) {
            float v[8];
            state_values<KIND>(load_codes(codes + i, n - i), scale[i / QC_STATE_BLOCK], v);
            store8(out + i, n - i, v);
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

template <class P, class G, class S, bool MASTER>
__global__ void __launch_bounds__(kThreads)
k_adamw(Tables l, P* const* __restrict__ params, G* const* __restrict__ grads, float* __restrict__ master, S st,
        AdamwStep step) {
    constexpr bool WIDE = std::is_same<S, Wide>::value;
    const Rates k = rates_of(step);
    const int64_t segs = (l.n + kSeg - 1) / kSeg;
    for (int64_t j = blockIdx.x; j < segs; j += gridDim.x) {
        int32_t lo, hi;
        tensors_of(l, j, lo, hi);
#pragma unroll 1
        for (int c = 0; c < kPasses; ++c) {
            const int64_t i = j * kSeg + c * kPass + threadIdx.x * kEach, left = l.n - i;
            float m[8] = {}, v[8] = {}, p[8] = {}, g[8] = {};
            Span at{lo, 0, false};
            if (left > 0) {
                if constexpr (WIDE) {
                    load8(st.m + i, left, m);
                    load8(st.v + i, left, v);
                } else {
                    state_values<QC_STATE_M>(load_codes(st.mc + i, left), st.ms[i / QC_STATE_BLOCK], m);
                    state_values<QC_STATE_R>(load_codes(st.rc + i, left), st.rs[i / QC_STATE_BLOCK], v);
                }
                if (MASTER) load8(master + i, left, p);
                at = span_of(l, lo, hi, i);
                load_span(l, grads, at, hi, i, g);
                if (!MASTER) load_span(l, params, at, hi, i, p);
            }
            float r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = g[e] * k.scale, old = WIDE ? v[e] : v[e] * v[e];
                m[e] = __builtin_fmaf(m[e], step.beta1, x * step.rest1);
                v[e] = __builtin_fmaf(old, step.beta2, x * x * step.rest2);
                r[e] = sqrtf(v[e]);
                const float den = __builtin_fmaf(r[e], k.root, step.eps);
                p[e] = p[e] * k.decay - k.rate * m[e] / den;
            }
            if constexpr (WIDE) {
                if (left > 0) {
                    store8(st.m + i, left, m);
                    store8(st.v + i, left, v);
                }
            } else {
                // every lane of the wave takes part; those past the end hold zeros
                const uint32_t u = (uint32_t)i * kDitherElem + k.t * kDitherStep;
                float ms, rs;
                const u32x2 mw = state_codes<QC_STATE_M>(m, u, kDitherElem, ms);
                const u32x2 rw = state_codes<QC_STATE_R>(r, u, kDitherElem, rs);
                if (left > 0) {
                    store_codes(st.mc + i, left, mw);
                    store_codes(st.rc + i, left, rw);
                    if ((threadIdx.x & 31) == 0) {
                        st.ms[i / QC_STATE_BLOCK] = ms;
                        st.rs[i / QC_STATE_BLOCK] = rs;
                    }
                }
            }
            if (left > 0) {
                if (MASTER) store8(master + i, left, p);
                store_span(l, params, at, hi, i, p);
            }
        }
    }
}

// ------------------------------------------------------------------- norm
// Squares are summed in 64 bits, so none overflows or vanishes.  Each block
// takes every gridDim-th segment and leaves its sum; a second kernel adds those
// up, always in the same order.
constexpr int kNormBlocks = 2048;

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if (lane_id() == 0) lds[wave_id()] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <class G>
__global__ void __launch_bounds__(kThreads)
k_norm_parts(Tables l, G* const* __restrict__ grads, double* __restrict__ parts) {
    __shared__ double lds[4];
    const int64_t segs = (l.n + kSeg - 1) / kSeg;
    double sum = 0.0;
    for (int64_t j = blockIdx.x; j < segs; j += gridDim.x) {
        int32_t lo, hi;
        tensors_of(l, j, lo, hi);
#pragma unroll
        for (int c = 0; c < kPasses; ++c) {
            const int64_t i = j * kSeg + c * kPass + threadIdx.x * kEach;
            if (i < l.n) {
                float g[8];
                load_span(l, grads, span_of(l, lo, hi, i), hi, i, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)g[e], (double)g[e], sum);
            }
        }
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads)
k_norm_join(const double* __restrict__ parts, int blocks, double max_norm, float* __restrict__ out) {
    __shared__ double lds[4];
    double sum = 0.0;
    for (int b = threadIdx.x; b < blocks; b += kThreads) sum += parts[b];
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum), c = max_norm / norm;
        out[0] = (float)norm;
        // an infinite norm clips with a NaN, not with zero, so that it is seen
        out[1] = norm - norm == 0.0 ? (float)(c < 1.0 ? c : 1.0) : __uint_as_float(0x7FC00000u);
    }
}

int norm_blocks(int64_t n) {
    const int64_t segs = (n + kSeg - 1) / kSeg;
    return (int)(segs < kNormBlocks ? segs : kNormBlocks);
}

unsigned grid_of(int64_t n, int64_t each) {
    const int64_t g = (n + each - 1) / each;
    return (unsigned)(g < kMaxBlocks ? g : kMaxBlocks);
}

Tables tables_of(const ListSrc& l) { return Tables{l.offsets, l.seg_first, l.ntensors, l.n}; }

template <class P, class G, class S, bool MASTER>
hipError_t launch_step(const AdamwList& l, const S& st, const AdamwStep& s, hipStream_t stream) {
    hipLaunchKernelGGL((k_adamw<P, G, S, MASTER>), dim3(grid_of(l.grads.n, kSeg)), dim3(kThreads), 0, stream,
                       tables_of(l.grads), reinterpret_cast<P* const*>(l.params),
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

int64_t grad_norm_workspace(int64_t n) { return 8 * (int64_t)norm_blocks(n); }

hipError_t launch_grad_norm(const ListSrc& l, bool bf16, double max_norm, void* workspace, float* out,
                            hipStream_t stream) {
    const int blocks = norm_blocks(l.n);
    double* parts = static_cast<double*>(workspace);
    auto xs = const_cast<void* const*>(reinterpret_cast<const void* const*>(l.xs));
    if (bf16)
        hipLaunchKernelGGL(k_norm_parts<BF16>, dim3(blocks), dim3(kThreads), 0, stream, tables_of(l),
                           reinterpret_cast<BF16* const*>(xs), parts);
    else
        hipLaunchKernelGGL(k_norm_parts<float>, dim3(blocks), dim3(kThreads), 0, stream, tables_of(l),
                           reinterpret_cast<float* const*>(xs), parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_norm_join, dim3(1), dim3(kThreads), 0, stream, parts, blocks, max_norm, out);
    return hipGetLastError();
}

}  // namespace qc
