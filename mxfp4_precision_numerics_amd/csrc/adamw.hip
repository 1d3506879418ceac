// adamw.hip - an AdamW step over any number of tensors for gfx950, moments in 32 bits or in 8.
//
//   g = grad min(1, max / (norm + 1e-6)),  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - rate decay) - rate / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Every value is read once and written once: HBM bounds it.  All tensors form one
// list of chunks of MXQ_CLIP_CHUNK elements (no chunk crosses a tensor), one block
// each, so that one launch serves any number of tensors of any size.
//
// 8-bit moments.  16 lanes hold a block of 128 elements, 8 each: the largest
// magnitude is four steps within a DPP row.  The scale is the block's own
// binary32 number, so that what all its elements share is kept exactly.  v takes
// E5M2 with rounding by chance: of 32768 elements whose gradients are normal
// deviates, after 4000 steps with beta2 = 0.999, sqrt(v) is off by 16% (rms) and
// by -1% in the mean; rounded to nearest in E4M3 or E5M2 it is off by 14-18%, but where half of them
// shrink by 4 it stays 3.4 times too large for good, 0.99 by chance.  E4M3 in
// place of E5M2 leaves 11%, but next to an element 1000 times larger (an
// outlier channel) its least code is 2.8 times too large in the mean, E5M2's 0.99.
#include "common.h"
#include "dense_launch.h"

namespace mxq {
namespace {

constexpr int NT = 256;
constexpr int64_t CH = MXQ_CLIP_CHUNK;
constexpr int EACH = 8, PASS = NT * EACH, PASSES = (int)(CH / PASS);

// What is the same for every element.
struct Step {
    float b1, c1, b2, c2;   // beta, 1 - beta
    float eps, decay;       // rate * weight decay
    float rate, root;       // rate / (1 - b1^t), 1 / sqrt(1 - b2^t)
    uint32_t word;
};
struct AdamwCall {
    Step s;
    double rate, beta1, beta2, weight_decay;
    float max_norm;
    int64_t step;
    const float *rate_at, *norm;
    const int64_t* step_at;
    uint64_t seed;
};

__host__ __device__ inline void set_step(Step& s, double rate, double b1, double b2, double wd, int64_t step, uint64_t seed) {
    s.rate = (float)(rate / (1.0 - pow(b1, (double)step)));
    s.root = (float)(1.0 / sqrt(1.0 - pow(b2, (double)step)));
    s.decay = (float)(rate * wd);
    uint64_t x = seed + (uint64_t)step * 0x9E3779B97F4A7C15u;
    x = (x ^ x >> 30) * 0xBF58476D1CE4E5B9u;
    x = (x ^ x >> 27) * 0x94D049BB133111EBu;
    s.word = (uint32_t)(x ^ x >> 31);
}

__device__ __forceinline__ uint32_t mixed(uint32_t r) {
    r = (r ^ r >> 16) * 0x85EBCA6Bu;
    r = (r ^ r >> 13) * 0xC2B2AE35u;
    return r ^ r >> 16;
}

// Vectors at their elements' alignment: gfx950 loads and stores them whole at any address.
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2b __attribute__((ext_vector_type(2), aligned(1)));
// The tensors' addresses come out of memory, where the compiler cannot see that they are global ones.
#define MXQ_GLOBAL __attribute__((address_space(1)))
template <class T> __device__ __forceinline__ const MXQ_GLOBAL T* from(const void* p, int64_t e) {
    return (const MXQ_GLOBAL T*)(uintptr_t)p + e;
}
template <class T> __device__ __forceinline__ MXQ_GLOBAL T* to(void* p, int64_t e) { return (MXQ_GLOBAL T*)(uintptr_t)p + e; }

__device__ __forceinline__ float bf(uint32_t u) { return as_float(u << 16); }
__device__ __forceinline__ uint32_t to_bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t two_bf(float a, float b) { return to_bf(a) | to_bf(b) << 16; }

// EACH values of a type: as they lie in memory.
template <int SRC> struct Raw;
template <> struct Raw<MXQ_SRC_F32> {
    u4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        const auto q = (const MXQ_GLOBAL u4*)from<float>(p, e);
        a = __builtin_nontemporal_load(q);
        b = __builtin_nontemporal_load(q + 1);
    }
    __device__ __forceinline__ void load_some(const void* p, int64_t e, int n) {
        a = b = u4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) (k < 4 ? a : b)[k & 3] = *from<uint32_t>(p, e + k);
    }
    __device__ __forceinline__ float at(int k) const { return as_float((k < 4 ? a : b)[k & 3]); }
    static __device__ __forceinline__ void store(void* p, int64_t e, const float (&f)[EACH]) {
        const auto q = (MXQ_GLOBAL u4*)to<float>(p, e);
        __builtin_nontemporal_store(u4{as_uint(f[0]), as_uint(f[1]), as_uint(f[2]), as_uint(f[3])}, q);
        __builtin_nontemporal_store(u4{as_uint(f[4]), as_uint(f[5]), as_uint(f[6]), as_uint(f[7])}, q + 1);
    }
    static __device__ __forceinline__ void store1(void* p, int64_t e, float f) { *to<float>(p, e) = f; }
};
template <> struct Raw<MXQ_SRC_BF16> {
    u4h a;
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        a = __builtin_nontemporal_load((const MXQ_GLOBAL u4h*)from<uint16_t>(p, e));
    }
    __device__ __forceinline__ void load_some(const void* p, int64_t e, int n) {
        a = u4h{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) a[k >> 1] |= (uint32_t)*from<uint16_t>(p, e + k) << (k & 1 ? 16 : 0);
    }
    __device__ __forceinline__ float at(int k) const { return k & 1 ? as_float(a[k >> 1] & 0xFFFF0000u) : bf(a[k >> 1]); }
    static __device__ __forceinline__ void store(void* p, int64_t e, const float (&f)[EACH]) {
        __builtin_nontemporal_store(u4h{two_bf(f[0], f[1]), two_bf(f[2], f[3]), two_bf(f[4], f[5]), two_bf(f[6], f[7])},
                                    (MXQ_GLOBAL u4h*)to<uint16_t>(p, e));
    }
    static __device__ __forceinline__ void store1(void* p, int64_t e, float f) { *to<uint16_t>(p, e) = (uint16_t)to_bf(f); }
};
struct Codes {
    u2b a;
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        a = __builtin_nontemporal_load((const MXQ_GLOBAL u2b*)from<uint8_t>(p, e));
    }
    __device__ __forceinline__ void load_some(const void* p, int64_t e, int n) {
        a = u2b{0u, 0u};
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) a[k >> 2] |= (uint32_t)*from<uint8_t>(p, e + k) << 8 * (k & 3);
    }
};

// The largest value of a row of 16 lanes, in each of them.
template <int CTRL> __device__ __forceinline__ float row_step(float v) {
    const float o = as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_uint(v), CTRL, 0xF, 0xF, false));
    return v > o ? v : o;
}
__device__ __forceinline__ float row_max(float v) {
    v = row_step<0x128>(v);  // row_ror:8, 4, 2, 1
    v = row_step<0x124>(v);
    v = row_step<0x122>(v);
    return row_step<0x121>(v);
}
// max over finite magnitudes
__device__ __forceinline__ float widened(float amax, float x) {
    const float a = __builtin_fabsf(x);
    return a > amax && a < __builtin_inff() ? a : amax;
}

// x / d rounded to nearest, from the rounded reciprocal of d: its product with x
// and one correction by the remainder.  Codes fall at a value next to a border by
// the last bit, and with the largest of a block the next step's scale: moments and quotients
// are therefore the plain sequence of binary32 operations, each rounded, that
// any program gets for the definition.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float q = x * inv;
    return __builtin_fabsf(x) == __builtin_inff() ? x : fmaf(fmaf(-q, d, x), inv, q);
}
// v / scale to a value of E5M2, rounded up by u / 2^16 against what is cut off.
__device__ __forceinline__ float chanced(float y, uint32_t u) {
    const float c = y < 57344.0f ? y : 57344.0f;
    const int e = (int)(as_uint(c) >> 23) - 129;  // of the step: two bits below the leading one ...
    const int s = e > -16 ? e : -16;              // ... but no smaller than 2^-16
    const float r = __builtin_amdgcn_ldexpf(floorf(__builtin_amdgcn_ldexpf(c, -s) + (float)u * 0x1p-16f), s);
    const float top = r < 57344.0f ? r : 57344.0f;
    const float some = c > 0.0f && top == 0.0f ? 0x1p-16f : top;
    return y != y ? y : some;
}

// sqrt of v >= 0, subnormal ones scaled first.
__device__ __forceinline__ float root_of(float v) {
    const bool small = v < 0x1p-96f;
    const float r = __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v);
    return small ? r * 0x1p-32f : r;
}

template <bool EIGHT, int P, int G> struct Group {
    Raw<P> p;
    Raw<G> g;
    typename std::conditional<EIGHT, Codes, Raw<MXQ_SRC_F32>>::type m, v;
    float sm, sv;
    __device__ __forceinline__ void load(const mxq_adamw_tensor& t, int64_t e, int n) {
        if (n >= EACH) {
            p.load(t.param, e); g.load(t.grad, e); m.load(t.m, e); v.load(t.v, e);
        } else {
            p.load_some(t.param, e, n); g.load_some(t.grad, e, n); m.load_some(t.m, e, n); v.load_some(t.v, e, n);
        }
        if constexpr (EIGHT) {
            sm = n > 0 ? *from<float>(t.m_scale, e / MXQ_STATE_BLOCK) : 0.0f;
            sv = n > 0 ? *from<float>(t.v_scale, e / MXQ_STATE_BLOCK) : 0.0f;
        }
    }
    __device__ __forceinline__ void step(const mxq_adamw_tensor& t, const Step& s, float coef, int64_t e, int n) const {
        float nm[EACH], nv[EACH], np[EACH];
        if constexpr (EIGHT) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)m.a[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)m.a[h], true);
                const auto c = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.a[h], false), d = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.a[h], true);
                nm[4 * h] = a[0] * sm; nm[4 * h + 1] = a[1] * sm; nm[4 * h + 2] = b[0] * sm; nm[4 * h + 3] = b[1] * sm;
                nv[4 * h] = c[0] * sv; nv[4 * h + 1] = c[1] * sv; nv[4 * h + 2] = d[0] * sv; nv[4 * h + 3] = d[1] * sv;
            }
        } else {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                nm[k] = m.at(k);
                nv[k] = v.at(k);
            }
        }
        const float decay = t.decay ? s.decay : 0.0f;
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const float x = g.at(k) * coef;
            nm[k] = s.b1 * nm[k] + s.c1 * x;  // each product rounded: see quotient()
            nv[k] = s.b2 * nv[k] + s.c2 * x * x;
            const float w = p.at(k);
            np[k] = fmaf(-s.rate * nm[k], __builtin_amdgcn_rcpf(fmaf(root_of(nv[k]), s.root, s.eps)), fmaf(-decay, w, w));
        }
        if (n >= EACH) {
            Raw<P>::store(t.param, e, np);
            if (t.copy) Raw<MXQ_SRC_BF16>::store(t.copy, e, np);
        } else {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                if (k >= n) continue;
                Raw<P>::store1(t.param, e + k, np[k]);
                if (t.copy) Raw<MXQ_SRC_BF16>::store1(t.copy, e + k, np[k]);
            }
        }
        if constexpr (EIGHT) {
            float am = 0.0f, av = 0.0f;
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                if (k < n) {
                    am = widened(am, nm[k]);
                    av = widened(av, nv[k]);
                }
            am = row_max(am);
            av = row_max(av);
            const float tm = am * (1.0f / 448.0f), tv = av * (1.0f / 57344.0f);
            const float zm = tm > 0x1p-120f ? tm : 0x1p-120f, zv = tv > 0x1p-120f ? tv : 0x1p-120f;
            const float im = 1.0f / zm, iv = 1.0f / zv;
            if (n <= 0) return;
            const uint64_t pair = ((uint64_t)t.first * CH + (uint64_t)e) / 2;
            const uint32_t word = s.word ^ (uint32_t)(pair >> 32) * 0x9E3779B1u;
            uint32_t cm[EACH / 2], cv[EACH / 2];
#pragma unroll
            for (int k = 0; k < EACH / 2; ++k) {
                const uint32_t r = mixed(((uint32_t)pair + k) ^ word);  // a block's pairs share their high word
                cm[k] = cast2_sat_f32<E4M3>(quotient(nm[2 * k], zm, im), quotient(nm[2 * k + 1], zm, im));
                cv[k] = cast2_sat_f32<E5M2>(chanced(quotient(nv[2 * k], zv, iv), r & 0xFFFFu),
                                              chanced(quotient(nv[2 * k + 1], zv, iv), r >> 16));
            }
            if (threadIdx.x % (MXQ_STATE_BLOCK / EACH) == 0) {
                *to<float>(t.m_scale, e / MXQ_STATE_BLOCK) = zm;
                *to<float>(t.v_scale, e / MXQ_STATE_BLOCK) = zv;
            }
            const auto om = to<uint8_t>(t.m, e), ov = to<uint8_t>(t.v, e);
            if (n >= EACH) {
                __builtin_nontemporal_store(u2b{cm[0] | cm[1] << 16, cm[2] | cm[3] << 16}, (MXQ_GLOBAL u2b*)om);
                __builtin_nontemporal_store(u2b{cv[0] | cv[1] << 16, cv[2] | cv[3] << 16}, (MXQ_GLOBAL u2b*)ov);
            } else {
#pragma unroll
                for (int k = 0; k < EACH; ++k) {
                    if (k >= n) continue;
                    om[k] = (uint8_t)(cm[k >> 1] >> 8 * (k & 1));
                    ov[k] = (uint8_t)(cv[k >> 1] >> 8 * (k & 1));
                }
            }
        } else if (n >= EACH) {
            Raw<MXQ_SRC_F32>::store(t.m, e, nm);
            Raw<MXQ_SRC_F32>::store(t.v, e, nv);
        } else {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                if (k >= n) continue;
                Raw<MXQ_SRC_F32>::store1(t.m, e + k, nm[k]);
                Raw<MXQ_SRC_F32>::store1(t.v, e + k, nv[k]);
            }
        }
    }
};

template <bool EIGHT, int P, int G>
__device__ __forceinline__ void chunk(const mxq_adamw_tensor& t, const Step& s, float coef, int64_t e0) {
    const int64_t left = t.numel - e0;
    const int n = (int)(left < CH ? left : CH), at = threadIdx.x * EACH;
    constexpr int HELD = EIGHT ? PASSES : 2;
    static_assert(PASSES % HELD == 0, "passes");
    for (int p0 = 0; p0 < PASSES && p0 * PASS < n; p0 += HELD) {
        Group<EIGHT, P, G> held[HELD];
#pragma unroll
        for (int p = 0; p < HELD; ++p) held[p].load(t, e0 + (p0 + p) * PASS + at, n - (p0 + p) * PASS - at);
#pragma unroll
        for (int p = 0; p < HELD; ++p) held[p].step(t, s, coef, e0 + (p0 + p) * PASS + at, n - (p0 + p) * PASS - at);
    }
}

template <bool EIGHT>
__global__ void __launch_bounds__(NT) k_adamw(const mxq_adamw_tensor* __restrict__ ts, const int32_t* __restrict__ chunk_of,
                                              int64_t first, const AdamwCall c) {
    const int64_t i = first + blockIdx.x;
    const mxq_adamw_tensor t = ts[chunk_of[i]];
    Step s = c.s;
    if (c.rate_at || c.step_at) {
        __shared__ Step shared;
        if (threadIdx.x == 0) {
            set_step(s, c.rate_at ? (double)*c.rate_at : c.rate, c.beta1, c.beta2, c.weight_decay, c.step_at ? *c.step_at : c.step,
                     c.seed);
            shared = s;
        }
        __syncthreads();
        s = shared;
    }
    float coef = 1.0f;
    if (c.norm) {
        const float q = 1.0f / (*c.norm + 1e-6f) * c.max_norm;
        coef = q > 1.0f ? 1.0f : q;  // a NaN norm stays NaN
    }
    const int64_t e0 = (i - t.first) * CH;
    if (t.param_src == MXQ_SRC_F32) {
        if (t.grad_src == MXQ_SRC_F32) chunk<EIGHT, MXQ_SRC_F32, MXQ_SRC_F32>(t, s, coef, e0);
        else chunk<EIGHT, MXQ_SRC_F32, MXQ_SRC_BF16>(t, s, coef, e0);
    } else {
        if (t.grad_src == MXQ_SRC_F32) chunk<EIGHT, MXQ_SRC_BF16, MXQ_SRC_F32>(t, s, coef, e0);
        else chunk<EIGHT, MXQ_SRC_BF16, MXQ_SRC_BF16>(t, s, coef, e0);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t st) {
    AdamwCall c{};
    c.s.b1 = (float)a.beta1; c.s.c1 = (float)(1.0 - a.beta1);
    c.s.b2 = (float)a.beta2; c.s.c2 = (float)(1.0 - a.beta2);
    c.s.eps = (float)a.eps;
    set_step(c.s, a.rate, a.beta1, a.beta2, a.weight_decay, a.step, a.seed);
    c.rate = a.rate; c.beta1 = a.beta1; c.beta2 = a.beta2; c.weight_decay = a.weight_decay; c.max_norm = (float)a.max_norm;
    c.step = a.step;
    c.rate_at = a.rate_at; c.norm = a.norm; c.step_at = a.step_at;
    c.seed = a.seed;
    for (int64_t k = 0; k < a.chunks; k += LAUNCH_THREADS / NT) {
        const unsigned n = (unsigned)(a.chunks - k < LAUNCH_THREADS / NT ? a.chunks - k : LAUNCH_THREADS / NT);
        if (a.states == MXQ_STATE_8BIT) k_adamw<true><<<n, NT, 0, st>>>(a.tensors, a.chunk_of, k, c);
        else k_adamw<false><<<n, NT, 0, st>>>(a.tensors, a.chunk_of, k, c);
    }
    return hipGetLastError();
}

}  // namespace mxq
