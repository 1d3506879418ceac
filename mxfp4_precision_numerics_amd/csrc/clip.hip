// clip.hip - clipping by the global gradient norm for gfx950:
// norm = sqrt(sum over all tensors of g^2), out = g * min(1, max / (norm + 1e-6)).
//
// The norm needs every element before any output is known, so the tensors are
// read twice: bytes = 2 reads + 1 write.  All tensors form one list of chunks
// of MXQ_CLIP_CHUNK elements (no chunk crosses a tensor), so two or three
// launches serve any number of tensors of any size.
//
// The second pass runs one block per chunk (16 KiB of bf16) with nontemporal
// loads and stores: 1.88 GB scaled in 598 us; 2048 blocks that loop over the
// chunks took 677 us, with plain loads 701.  Both passes 909 us (6.2 TB/s), 930
// with the products in binary32.
#include "common.h"
#include "train_launch.h"

namespace mxq {
namespace {

constexpr int NT = 256;
constexpr int64_t CH = MXQ_CLIP_CHUNK;

// Sum of the block's values, the same for every thread and from run to run.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < NT / 64; ++i) s += part[i];
    return s;
}

__device__ __forceinline__ float bf(uint16_t u) { return as_float((uint32_t)u << 16); }
// Round to nearest even; a NaN stays a (quiet) NaN.
__device__ __forceinline__ uint16_t to_bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// Elements before the first 16-byte boundary at or after p (at most n).
template <int ESZ> __device__ __forceinline__ int head_of(const uint8_t* p, int n) {
    const int h = (int)((16 - ((uintptr_t)p & 15)) & 15) / ESZ;
    return h < n ? h : n;
}

template <int ESZ> __device__ __forceinline__ float load1(const uint8_t* p, int i) {
    if constexpr (ESZ == 2) return bf(((const uint16_t*)p)[i]);
    else return ((const float*)p)[i];
}
// Squares in binary64: an element of any size keeps its place in the norm
// (in binary32 those above 2^64 or below 2^-75 would leave it).
__device__ __forceinline__ double sq(float f, double s) { return fma((double)f, (double)f, s); }
template <int ESZ> __device__ __forceinline__ double sq16(const uint4 v, double s) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (ESZ == 2) s = sq(as_float(u[k] & 0xFFFF0000u), sq(as_float(u[k] << 16), s));
        else s = sq(as_float(u[k]), s);
    }
    return s;
}

template <int ESZ> __device__ __forceinline__ double sum_sq(const uint8_t* p, int n, double s) {
    const int head = head_of<ESZ>(p, n);
    if ((int)threadIdx.x < head) s = sq(load1<ESZ>(p, threadIdx.x), s);
    const uint8_t* b = p + head * ESZ;
    constexpr int VE = 16 / ESZ;
    const int nv = (n - head) / VE;
#pragma unroll 4
    for (int i = threadIdx.x; i < nv; i += NT) s = sq16<ESZ>(ld_nt16(b + (size_t)i * 16), s);
    const int t = head + nv * VE + threadIdx.x;
    if (t < n) s = sq(load1<ESZ>(p, t), s);
    return s;
}

// The coefficient and its products are binary64 too: for a norm beyond 1e38 a
// binary32 coefficient is subnormal or zero, where the products are not (and
// elsewhere its own rounding would add half a step to theirs).
__device__ __forceinline__ float scaled(float f, double c) { return (float)((double)f * c); }

template <int ESZ> __device__ __forceinline__ uint4 scale16(const uint4 v, double c) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (ESZ == 2)
            r[k] = (uint32_t)to_bf(scaled(as_float(u[k] << 16), c)) |
                   (uint32_t)to_bf(scaled(as_float(u[k] & 0xFFFF0000u), c)) << 16;
        else
            r[k] = as_uint(scaled(as_float(u[k]), c));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int ESZ> __device__ __forceinline__ void store1(uint8_t* p, int i, float f) {
    if constexpr (ESZ == 2) ((uint16_t*)p)[i] = to_bf(f);
    else ((float*)p)[i] = f;
}

// A chunk on its way from p to o: what lies on 16-byte boundaries of both in
// registers, loaded before the coefficient is known.
template <int ESZ> struct Held {
    static constexpr int VE = 16 / ESZ, NV = (int)(CH / VE / NT);
    uint4 v[NV];
    int head, nv;
    __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* o, int n) {
        head = n;
        nv = 0;
        if ((((uintptr_t)p ^ (uintptr_t)o) & 15) == 0) {  // both reach a boundary together
            head = head_of<ESZ>(p, n);
            nv = (n - head) / VE;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i < nv) v[k] = ld_nt16(p + head * ESZ + (size_t)i * 16);
        }
    }
    __device__ __forceinline__ void store(const uint8_t* p, uint8_t* o, int n, double c) const {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = threadIdx.x + k * NT;
            if (i < nv) st_nt16(o + head * ESZ + (size_t)i * 16, scale16<ESZ>(v[k], c));
        }
        for (int i = threadIdx.x; i < head; i += NT) store1<ESZ>(o, i, scaled(load1<ESZ>(p, i), c));
        for (int i = head + nv * VE + threadIdx.x; i < n; i += NT) store1<ESZ>(o, i, scaled(load1<ESZ>(p, i), c));
    }
};

__global__ void __launch_bounds__(NT) k_clip_norm(const mxq_clip_tensor* __restrict__ ts,
                                                  const int32_t* __restrict__ chunk_of, int64_t chunks,
                                                  double* __restrict__ parts) {
    __shared__ double part[NT / 64];
    double acc = 0.0;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const mxq_clip_tensor t = ts[chunk_of[c]];
        const int64_t e0 = (c - t.first) * CH;
        const int n = (int)(t.numel - e0 < CH ? t.numel - e0 : CH);
        const uint8_t* p = (const uint8_t*)t.in;
        acc = t.src == MXQ_SRC_BF16 ? sum_sq<2>(p + e0 * 2, n, acc) : sum_sq<4>(p + e0 * 4, n, acc);
    }
    const double s = block_sum(acc, part);
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

// norm and coefficient from the partial sums, the same in every thread.
__device__ __forceinline__ double coef_of(const double* parts, int nparts, float max_norm, double* part, double& n2) {
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += NT) s += parts[i];
    n2 = sqrt(block_sum(s, part));
    const double q = (double)max_norm / (n2 + 1e-6);
    return q > 1.0 ? 1.0 : q;  // a NaN norm stays NaN
}

__global__ void __launch_bounds__(NT) k_clip_coef(double* parts, int nparts, float max_norm, float* norm) {
    __shared__ double part[NT / 64];
    double n2;
    const double coef = coef_of(parts, nparts, max_norm, part, n2);  // every part is read before its last barrier
    if (threadIdx.x == 0) {
        *norm = (float)n2;
        parts[0] = coef;
    }
}

// One block per chunk.  nparts > 0: the block adds the partial sums up itself
// while its chunk is on the way; 0: k_clip_coef has left the coefficient in
// parts[0].  A coefficient of one leaves tensors clipped in place alone.
template <int ESZ>
__device__ __forceinline__ void scale_chunk(const mxq_clip_tensor& t, int64_t c, const double* parts, int nparts,
                                            float max_norm, float* norm, double* part) {
    const int64_t e0 = (c - t.first) * CH;
    const int n = (int)(t.numel - e0 < CH ? t.numel - e0 : CH);
    const uint8_t* p = (const uint8_t*)t.in + e0 * ESZ;
    uint8_t* o = (uint8_t*)t.out + e0 * ESZ;
    Held<ESZ> h;
    double coef;
    if (nparts) {
        h.load(p, o, n);
        double n2;
        coef = coef_of(parts, nparts, max_norm, part, n2);
        if (c == 0 && threadIdx.x == 0) *norm = (float)n2;
        if (coef == 1.0 && p == o) return;
    } else {
        coef = parts[0];
        if (coef == 1.0 && p == o) return;
        h.load(p, o, n);
    }
    h.store(p, o, n, coef);
}

__global__ void __launch_bounds__(NT) k_clip_scale(const mxq_clip_tensor* __restrict__ ts,
                                                   const int32_t* __restrict__ chunk_of, int64_t first,
                                                   const double* __restrict__ parts, int nparts, float max_norm,
                                                   float* __restrict__ norm) {
    __shared__ double part[NT / 64];
    const int64_t c = first + blockIdx.x;
    const mxq_clip_tensor t = ts[chunk_of[c]];
    if (t.src == MXQ_SRC_BF16) scale_chunk<2>(t, c, parts, nparts, max_norm, norm, part);
    else scale_chunk<4>(t, c, parts, nparts, max_norm, norm, part);
}

}  // namespace

// Up to OWN_SUM chunks every block adds the partial sums up itself, which saves
// a launch (3922 chunks 34.6 us of kernels against 38.8, 1263 chunks 14.8 against
// 17.0); above, where it would no longer gain (7361: 65.2 / 66.6), one more launch
// does it once.
constexpr int64_t OWN_SUM = 4096;

hipError_t launch_clip(const mxq_clip_tensor* t, const int32_t* chunk_of, int64_t chunks, float max_norm, float* norm,
                       double* parts, hipStream_t st) {
    const int nb = (int)(chunks < MXQ_CLIP_PARTS ? (chunks ? chunks : 1) : MXQ_CLIP_PARTS);
    k_clip_norm<<<nb, NT, 0, st>>>(t, chunk_of, chunks, parts);
    const bool own = chunks <= OWN_SUM;
    if (!own || chunks == 0) k_clip_coef<<<1, NT, 0, st>>>(parts, nb, max_norm, norm);
    for (int64_t c = 0; c < chunks; c += LAUNCH_THREADS / NT) {
        const int64_t n = chunks - c < LAUNCH_THREADS / NT ? chunks - c : LAUNCH_THREADS / NT;
        k_clip_scale<<<(unsigned)n, NT, 0, st>>>(t, chunk_of, c, parts, own ? nb : 0, max_norm, norm);
    }
    return hipGetLastError();
}

}  // namespace mxq
