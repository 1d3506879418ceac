// adamw.hip - an AdamW step over any number of tensors for gfx950, moments in 32 bits or in 8.
//
//   g = grad min(1, max / (norm + 1e-6)),  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - rate decay) - rate / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Every value is read once and written once: HBM bounds it.  All tensors form one
// list of chunks of MXQ_CLIP_CHUNK elements (no chunk crosses a tensor), one block
// four or eight each, so that one launch serves any number of tensors of any size.  Blocks as short
// as that keep more loads on their way: 470 million elements, bf16 gradients and copies, 32-bit moments, 2.23
// ms with eight (5.9 TB/s), 2.37 with four, 2.42 with one; 8-bit moments 1.24-1.31 ms with four (5.8-6.1 TB/s), 1.39 with two, 1.42 with
// one, and 1.72 with eight, where a block's own start weighs.  5.5 million ragged ones (rows off the 16-byte
// boundaries), all in 32 bits: 30 us (5.1 TB/s).
//
// 8-bit moments.  32 lanes hold a block of 128 elements, 4 each: the largest
// magnitude is four steps within a DPP row and one across two.  The scale is the block's own
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
constexpr int EACH = 4, PASS = NT * EACH;  // elements of a lane, of a block, at a time
constexpr int LANES = MXQ_STATE_BLOCK / EACH;

// What is the same for every element.
struct Step {
    float b1, c1, b2, c2;   // beta, 1 - beta
    float eps, decay;       // rate * weight decay
    float rate, root;       // rate / (1 - b1^t), 1 / sqrt(lift (1 - b2^t))
    float lift;             // what v is multiplied with before its root
    uint32_t word;
};
// What gradients are taken times: `coef`, or, where it is not 0, `wide`.
struct Clip { float coef; double wide; };
struct AdamwCall {
    Step s;
    double rate, beta1, beta2, weight_decay, max_norm;
    int64_t step;
    const float *rate_at, *norm;
    const int64_t* step_at;
    uint64_t seed;
};

__host__ __device__ inline void set_step(Step& s, double rate, double b1, double b2, double wd, int64_t step, uint64_t seed) {
    s.rate = (float)(rate / (1.0 - pow(b1, (double)step)));
    s.root = (float)(1.0 / sqrt((double)s.lift * (1.0 - pow(b2, (double)step))));
    s.decay = (float)(rate * wd);
    uint64_t x = seed + (uint64_t)step * 0x9E3779B97F4A7C15u;  // SplitMix64 (Steele, Lea and Flood 2014)
    x = (x ^ x >> 30) * 0xBF58476D1CE4E5B9u;
    x = (x ^ x >> 27) * 0x94D049BB133111EBu;
    s.word = (uint32_t)(x ^ x >> 31);
}

// The clipping coefficient min(1, max_norm / (norm + 1e-6)) in binary32, as its products with the gradients are, wherever
// nothing on the way leaves the normal numbers.  Near their ends (norms or limits beyond 2^100, coefficients below 2^-100) a
// reciprocal or the coefficient would be subnormal or zero where the products are not: there both are binary64, as clip.hip's.
__device__ __forceinline__ Clip clip_of(const AdamwCall& c) {
    if (!c.norm) return {1.0f, 0.0};
    const float norm = *c.norm, most = (float)c.max_norm;
    const float q = 1.0f / (norm + 1e-6f) * most;
    if (norm > 0x1p100f || most > 0x1p100f || q < 0x1p-100f) {
        const double w = c.max_norm / ((double)norm + 1e-6);
        if (w < 1.0) return {0.0f, w};  // (of zero where w is)
        return {w >= 1.0 ? 1.0f : norm, 0.0};
    }
    return {q > 1.0f ? 1.0f : q, 0.0};  // a NaN norm stays NaN
}

// The finalizer of Appleby's MurmurHash3.
__device__ __forceinline__ uint32_t mixed(uint32_t r) {
    r = (r ^ r >> 16) * 0x85EBCA6Bu;
    r = (r ^ r >> 13) * 0xC2B2AE35u;
    return r ^ r >> 16;
}

// Vectors at their elements' alignment: gfx950 loads and stores them whole at any address.
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u1b __attribute__((aligned(1)));
// The tensors' addresses come out of memory, where the compiler cannot see that they are global ones.
#define MXQ_GLOBAL __attribute__((address_space(1)))
// An element is the block's first one, the same for all lanes, and a lane's own from there on.
struct At { int64_t first; uint32_t lane; };
__device__ __forceinline__ At operator+(At a, int k) { return {a.first, a.lane + (uint32_t)k}; }
__device__ __forceinline__ At scale_of(At a) { return {a.first / MXQ_STATE_BLOCK, a.lane / MXQ_STATE_BLOCK}; }
template <class T> __device__ __forceinline__ const MXQ_GLOBAL T* from(const void* p, At e) {
    return (const MXQ_GLOBAL T*)(uintptr_t)p + e.first + e.lane;
}
template <class T> __device__ __forceinline__ MXQ_GLOBAL T* to(void* p, At e) {
    return (MXQ_GLOBAL T*)(uintptr_t)p + e.first + e.lane;
}

__device__ __forceinline__ float bf(uint32_t u) { return as_float(u << 16); }
__device__ __forceinline__ uint32_t to_bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint32_t two_bf(float a, float b) { return to_bf(a) | to_bf(b) << 16; }

// EACH values of a type: as they lie in memory.
template <int SRC> struct Raw;
template <> struct Raw<MXQ_SRC_F32> {
    u4 a;
    __device__ __forceinline__ void load(const void* p, At e) {
        a = __builtin_nontemporal_load((const MXQ_GLOBAL u4*)from<float>(p, e));
    }
    __device__ __forceinline__ void load_some(const void* p, At e, int n) {
        a = u4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) a[k] = *from<uint32_t>(p, e + k);
    }
    __device__ __forceinline__ float at(int k) const { return as_float(a[k]); }
    static __device__ __forceinline__ void store(void* p, At e, const float (&f)[EACH]) {
        __builtin_nontemporal_store(u4{as_uint(f[0]), as_uint(f[1]), as_uint(f[2]), as_uint(f[3])},
                                    (MXQ_GLOBAL u4*)to<float>(p, e));
    }
    static __device__ __forceinline__ void store1(void* p, At e, float f) { *to<float>(p, e) = f; }
};
template <> struct Raw<MXQ_SRC_BF16> {
    u2h a;
    __device__ __forceinline__ void load(const void* p, At e) {
        a = __builtin_nontemporal_load((const MXQ_GLOBAL u2h*)from<uint16_t>(p, e));
    }
    __device__ __forceinline__ void load_some(const void* p, At e, int n) {
        a = u2h{0u, 0u};
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) a[k >> 1] |= (uint32_t)*from<uint16_t>(p, e + k) << (k & 1 ? 16 : 0);
    }
    __device__ __forceinline__ float at(int k) const { return k & 1 ? as_float(a[k >> 1] & 0xFFFF0000u) : bf(a[k >> 1]); }
    static __device__ __forceinline__ void store(void* p, At e, const float (&f)[EACH]) {
        __builtin_nontemporal_store(u2h{two_bf(f[0], f[1]), two_bf(f[2], f[3])}, (MXQ_GLOBAL u2h*)to<uint16_t>(p, e));
    }
    static __device__ __forceinline__ void store1(void* p, At e, float f) { *to<uint16_t>(p, e) = (uint16_t)to_bf(f); }
};
struct Codes {
    u1b a;
    __device__ __forceinline__ void load(const void* p, At e) {
        a = __builtin_nontemporal_load((const MXQ_GLOBAL u1b*)from<uint8_t>(p, e));
    }
    __device__ __forceinline__ void load_some(const void* p, At e, int n) {
        a = 0u;
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < n) a |= (uint32_t)*from<uint8_t>(p, e + k) << 8 * k;
    }
    static __device__ __forceinline__ void store(void* p, At e, uint32_t c) {
        __builtin_nontemporal_store(c, (MXQ_GLOBAL u1b*)to<uint8_t>(p, e));
    }
};

// The largest of a block's lanes (two rows of 16), in each of them.
template <int CTRL> __device__ __forceinline__ uint32_t row_step(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    static_assert(LANES == 32, "two rows of lanes");
    v = row_step<0x128>(v);  // row_ror:8, 4, 2, 1
    v = row_step<0x124>(v);
    v = row_step<0x122>(v);
    v = row_step<0x121>(v);
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // {even rows, odd rows}, each twice
    return r[0] > r[1] ? r[0] : r[1];
}
constexpr uint32_t INF = 0x7F800000u;

// x / d rounded to nearest, from a reciprocal of d that is off by an ulp at most: its product with x
// and one correction by the remainder.  Codes fall at a value next to a border by
// the last bit, and with the largest of a block the next step's scale: moments and quotients
// are therefore the sequence of binary32 operations, each rounded, that the
// header states and any program can repeat.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, d, x), inv, q);
}
// y = v / scale in [2^-14, F] to an E5M2 code, rounded up by u / 2^16 against what is
// cut off: 21 bits of the significand, whose top 16 u joins.
__device__ __forceinline__ uint32_t chanced(float y, uint32_t u) {
    return (as_uint(y) + ((u << 5) - (112u << 23))) >> 21;
}
// The same for any y >= 0 (above F: F; a NaN: a NaN), and not to zero unless y is.
__device__ __forceinline__ uint32_t chanced_any(float y, uint32_t u) {
    if (y != y) return 0x7Fu;
    if (y >= 57344.0f) return 0x7Bu;
    const uint32_t c = y < 0x1p-14f ? (uint32_t)floorf(fmaf(y, 0x1p16f, (float)u * 0x1p-16f)) : chanced(y, u);
    return c == 0u && y > 0.0f ? 1u : c;
}

template <bool EIGHT, int P, int G> struct Group {
    Raw<P> p;
    Raw<G> g;
    typename std::conditional<EIGHT, Codes, Raw<MXQ_SRC_F32>>::type m, v;
    float sm, sv;
    __device__ __forceinline__ void load(const mxq_adamw_tensor& t, At e, int n) {
        if (n >= EACH) {
            p.load(t.param, e); g.load(t.grad, e); m.load(t.m, e); v.load(t.v, e);
        } else {
            p.load_some(t.param, e, n); g.load_some(t.grad, e, n); m.load_some(t.m, e, n); v.load_some(t.v, e, n);
        }
        if constexpr (EIGHT) {
            sm = n > 0 ? *from<float>(t.m_scale, scale_of(e)) : 0.0f;
            sv = n > 0 ? *from<float>(t.v_scale, scale_of(e)) : 0.0f;
        }
    }
    __device__ __forceinline__ void step(const mxq_adamw_tensor& t, const Step& s, const Clip& c, At e, int n) const {
        float nm[EACH], nv[EACH], np[EACH];
        if constexpr (EIGHT) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)m.a, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)m.a, true);
            const auto c = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.a, false), d = __builtin_amdgcn_cvt_pk_f32_bf8((int)v.a, true);
            nm[0] = a[0] * sm; nm[1] = a[1] * sm; nm[2] = b[0] * sm; nm[3] = b[1] * sm;
            nv[0] = c[0] * sv; nv[1] = c[1] * sv; nv[2] = d[0] * sv; nv[3] = d[1] * sv;
        } else {
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                nm[k] = m.at(k);
                nv[k] = v.at(k);
            }
        }
        const float decay = t.decay ? s.decay : 0.0f;
        float gc[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) gc[k] = g.at(k) * c.coef;
        if (c.wide != 0.0)  // the same for all threads
#pragma unroll
            for (int k = 0; k < EACH; ++k) gc[k] = (float)((double)g.at(k) * c.wide);
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const float x = gc[k];
            nm[k] = s.b1 * nm[k] + s.c1 * x;  // each product rounded: see quotient()
            nv[k] = s.b2 * nv[k] + s.c2 * x * x;
            const float w = p.at(k);
            np[k] = fmaf(-s.rate * nm[k], __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_sqrtf(nv[k] * s.lift), s.root, s.eps)),
                         fmaf(-decay, w, w));
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
            // magnitudes as integers: what is not finite comes out above all numbers
            uint32_t am = 0u, av = 0u;
#pragma unroll
            for (int k = 0; k < EACH; ++k) {  // lanes past the end hold zeros
                const uint32_t x = as_uint(nm[k]) & 0x7FFFFFFFu, y = as_uint(nv[k]);
                am = x > am ? x : am;
                av = y > av ? y : av;
            }
            am = block_max(am);
            av = block_max(av);
            const bool finite = am < INF && av < INF;
            if (!__all(finite)) {  // the largest of the others
                uint32_t fm = 0u, fv = 0u;
#pragma unroll
                for (int k = 0; k < EACH; ++k) {
                    const uint32_t x = as_uint(nm[k]) & 0x7FFFFFFFu, y = as_uint(nv[k]) & 0x7FFFFFFFu;
                    fm = x > fm && x < INF ? x : fm;
                    fv = y > fv && y < INF ? y : fv;
                }
                am = block_max(fm);
                av = block_max(fv);
            }
            // the scale's definition: the reciprocal of the format's largest value is a constant, and a product rounded once more than
            // a quotient costs the codes nothing, as they are taken with the scale that is stored
            const float tm = as_float(am) * (1.0f / 448.0f), tv = as_float(av) * (1.0f / 57344.0f);
            const float zm = tm > 0x1p-120f ? tm : 0x1p-120f, zv = tv > 0x1p-120f ? tv : 0x1p-120f;
            const float im = __builtin_amdgcn_rcpf(zm), iv = __builtin_amdgcn_rcpf(zv);
            const uint64_t pair = ((uint64_t)t.first * CH + (uint64_t)e.first) / 2;  // a pass's pairs share its high word
            const uint32_t word = s.word ^ (uint32_t)(pair >> 32) * 0x9E3779B1u, low = (uint32_t)pair + e.lane / 2;
            float ym[EACH], yv[EACH];
            uint32_t least = INF;  // of numbers that are not negative, as integers
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                ym[k] = quotient(nm[k], zm, im);
                yv[k] = quotient(nv[k], zv, iv);
                least = as_uint(yv[k]) < least ? as_uint(yv[k]) : least;
            }
            uint32_t r[EACH / 2];
#pragma unroll
            for (int k = 0; k < EACH / 2; ++k) r[k] = mixed((low + k) ^ word);
            uint32_t cm, cv = 0u;
            if (__all(finite && least >= 113u << 23)) {
                float z[EACH];
#pragma unroll
                for (int k = 0; k < EACH; ++k) z[k] = __builtin_amdgcn_fmed3f(ym[k], -448.0f, 448.0f);
                cm = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
                cm = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], (int)cm, true);
#pragma unroll
                for (int k = 0; k < EACH; ++k) cv |= chanced(yv[k], k & 1 ? r[k >> 1] >> 16 : r[k >> 1] & 0xFFFFu) << 8 * k;
            } else {
                const auto one = [](float x, float y) { return as_uint(x) << 1 == INF << 1 ? x : y; };  // an infinity stays one
                cm = cast2_sat_f32<E4M3>(one(nm[0], ym[0]), one(nm[1], ym[1])) |
                     cast2_sat_f32<E4M3>(one(nm[2], ym[2]), one(nm[3], ym[3])) << 16;
#pragma unroll
                for (int k = 0; k < EACH; ++k)
                    cv |= chanced_any(one(nv[k], yv[k]), k & 1 ? r[k >> 1] >> 16 : r[k >> 1] & 0xFFFFu) << 8 * k;
            }
            if (n <= 0) return;
            if (threadIdx.x % LANES == 0) {
                *to<float>(t.m_scale, scale_of(e)) = zm;
                *to<float>(t.v_scale, scale_of(e)) = zv;
            }
            if (n >= EACH) {
                Codes::store(t.m, e, cm);
                Codes::store(t.v, e, cv);
            } else {
#pragma unroll
                for (int k = 0; k < EACH; ++k) {
                    if (k >= n) continue;
                    *to<uint8_t>(t.m, e + k) = (uint8_t)(cm >> 8 * k);
                    *to<uint8_t>(t.v, e + k) = (uint8_t)(cv >> 8 * k);
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

// Elements e0 .. e0 + n - 1 of a tensor.
template <bool EIGHT, int P, int G>
__device__ __forceinline__ void part(const mxq_adamw_tensor& t, const Step& s, const Clip& c, int64_t e0, int n) {
    const int at = (int)threadIdx.x * EACH;
    constexpr int HELD = EIGHT ? 2 : 1;  // passes whose loads are on their way together
    for (int p0 = 0; p0 < n; p0 += HELD * PASS) {
        Group<EIGHT, P, G> held[HELD];
#pragma unroll
        for (int p = 0; p < HELD; ++p) held[p].load(t, At{e0 + p0 + p * PASS, (uint32_t)at}, n - p0 - p * PASS - at);
#pragma unroll
        for (int p = 0; p < HELD; ++p) held[p].step(t, s, c, At{e0 + p0 + p * PASS, (uint32_t)at}, n - p0 - p * PASS - at);
    }
}

// `parts` blocks for each chunk.
template <bool EIGHT>
__global__ void __launch_bounds__(NT) k_adamw(const mxq_adamw_tensor* __restrict__ ts, const int32_t* __restrict__ chunk_of,
                                              int64_t first, int parts, const AdamwCall c) {
    const int64_t i = first + blockIdx.x / parts;
    const int size = (int)CH / parts;
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
    const Clip k = clip_of(c);
    const int64_t e0 = (i - t.first) * CH + (int64_t)(blockIdx.x % parts) * size, left = t.numel - e0;
    if (left <= 0) return;
    const int n = (int)(left < size ? left : size);
    if (t.param_src == MXQ_SRC_F32) {
        if (t.grad_src == MXQ_SRC_F32) part<EIGHT, MXQ_SRC_F32, MXQ_SRC_F32>(t, s, k, e0, n);
        else part<EIGHT, MXQ_SRC_F32, MXQ_SRC_BF16>(t, s, k, e0, n);
    } else {
        if (t.grad_src == MXQ_SRC_F32) part<EIGHT, MXQ_SRC_BF16, MXQ_SRC_F32>(t, s, k, e0, n);
        else part<EIGHT, MXQ_SRC_BF16, MXQ_SRC_BF16>(t, s, k, e0, n);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t st) {
    AdamwCall c{};
    c.s.b1 = (float)a.beta1; c.s.c1 = (float)(1.0 - a.beta1);
    c.s.b2 = (float)a.beta2; c.s.c2 = (float)(1.0 - a.beta2);
    c.s.eps = (float)a.eps;
    // A root takes a subnormal v for zero: up to 2^-63 / sqrt(1 - beta2^step) of the denominator, which is less than 2^-24 of eps
    // only from 2^-39 / sqrt(1 - beta2) on.
    c.s.lift = a.eps < 0x1p-34 || a.eps * sqrt(1.0 - a.beta2) < 0x1p-39 ? 0x1p32f : 1.0f;
    set_step(c.s, a.rate, a.beta1, a.beta2, a.weight_decay, a.step, a.seed);
    c.rate = a.rate; c.beta1 = a.beta1; c.beta2 = a.beta2; c.weight_decay = a.weight_decay; c.max_norm = a.max_norm;
    c.step = a.step;
    c.rate_at = a.rate_at; c.norm = a.norm; c.step_at = a.step_at;
    c.seed = a.seed;
    const int parts = a.states == MXQ_STATE_8BIT ? 4 : 8;
    const int64_t most = LAUNCH_THREADS / NT / parts;
    for (int64_t k = 0; k < a.chunks; k += most) {
        const unsigned n = (unsigned)(a.chunks - k < most ? a.chunks - k : most) * parts;
        if (a.states == MXQ_STATE_8BIT) k_adamw<true><<<n, NT, 0, st>>>(a.tensors, a.chunk_of, k, parts, c);
        else k_adamw<false><<<n, NT, 0, st>>>(a.tensors, a.chunk_of, k, parts, c);
    }
    return hipGetLastError();
}

}  // namespace mxq
