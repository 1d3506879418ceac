// moe.hip - the mixture-of-experts router and the movement of token rows to
// and from their experts, for gfx950.
//
// MoE FP4 page, "Kernels CUDA Otimizados": ragged per-expert token counts;
// "Metodologia": the rows that reach the experts' products are quantized.
#include "common.h"
#include "train_launch.h"

namespace mxq {
namespace {

// Reductions over the wave on DPP moves (row shifts, then the two row
// broadcasts), the result in every lane through a scalar register.
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t dpp_or0(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_u(v, dpp_or0<0x111, 0xF>(v));
    v = max_u(v, dpp_or0<0x112, 0xF>(v));
    v = max_u(v, dpp_or0<0x114, 0xF>(v));
    v = max_u(v, dpp_or0<0x118, 0xF>(v));
    v = max_u(v, dpp_or0<0x142, 0xA>(v));
    v = max_u(v, dpp_or0<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL, int ROWS> __device__ __forceinline__ float plus_dpp(float v) {
    return v + as_float(dpp_or0<CTRL, ROWS>(as_uint(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = plus_dpp<0x111, 0xF>(v);
    v = plus_dpp<0x112, 0xF>(v);
    v = plus_dpp<0x114, 0xF>(v);
    v = plus_dpp<0x118, 0xF>(v);
    v = plus_dpp<0x142, 0xA>(v);
    v = plus_dpp<0x143, 0xC>(v);
    return as_float((uint32_t)__builtin_amdgcn_readlane((int)as_uint(v), 63));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return as_float((uint32_t)__builtin_amdgcn_readlane((int)as_uint(v), lane));
}

template <int SRC> __device__ __forceinline__ float load_el(const void* p, int64_t i) {
    if constexpr (SRC == MXQ_SRC_BF16) return as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    else return ((const float*)p)[i];
}
__device__ __forceinline__ uint16_t to_bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// ---------------------------------------------------------------------------
// Router.  One wave per token; lane l holds experts l * NV .. l * NV + NV - 1,
// so that among equal logits the lowest lane, and in it the lowest slot, is
// the lowest expert.
// ---------------------------------------------------------------------------

// A logit as an unsigned key of the same order: -0 like +0, NaN above all; 0
// marks an expert that is taken or past the end (the key of -inf is larger).
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t u = as_uint(z + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return as_float((k >> 31) ? (k == 0xFFFFFFFFu ? 0x7FC00000u : (k & 0x7FFFFFFFu)) : ~k);
}

// The lane's NV logits of a row; VEC: rows, and so every lane's run, aligned to
// the run's size and E a multiple of NV.
template <int NV, int SRC, bool VEC>
__device__ __forceinline__ void load_run(const void* z, int64_t at, int E, int lane, float (&v)[NV]) {
    constexpr int BYTES = NV * (SRC == MXQ_SRC_BF16 ? 2 : 4);
    if constexpr (VEC && BYTES >= 4) {
        uint32_t w[BYTES / 4];
        if (lane * NV < E) {
            const uint8_t* p = (const uint8_t*)z + (at + lane * NV) * (BYTES / NV);
            if constexpr (BYTES == 4) w[0] = *(const uint32_t*)p;
            else if constexpr (BYTES == 8) { const uint2 c = *(const uint2*)p; w[0] = c.x; w[1] = c.y; }
            else
#pragma unroll
                for (int i = 0; i < BYTES / 16; ++i) {
                    const uint4 c = *(const uint4*)(p + 16 * i);
                    w[4 * i] = c.x; w[4 * i + 1] = c.y; w[4 * i + 2] = c.z; w[4 * i + 3] = c.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i) w[i] = 0u;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (SRC == MXQ_SRC_BF16) v[j] = as_float((j & 1) ? (w[j / 2] & 0xFFFF0000u) : (w[j / 2] << 16));
            else v[j] = as_float(w[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = lane * NV + j < E ? load_el<SRC>(z, at + lane * NV + j) : 0.0f;
    }
}
template <int NV, int SRC, bool VEC>
__device__ __forceinline__ void store_run(void* z, int64_t at, int E, int lane, const float (&v)[NV]) {
    constexpr int BYTES = NV * (SRC == MXQ_SRC_BF16 ? 2 : 4);
    if constexpr (VEC && BYTES >= 4) {
        if (lane * NV >= E) return;
        uint32_t w[BYTES / 4];
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) {
            if constexpr (SRC == MXQ_SRC_BF16) w[i] = (uint32_t)to_bf(v[2 * i]) | (uint32_t)to_bf(v[2 * i + 1]) << 16;
            else w[i] = as_uint(v[i]);
        }
        uint8_t* p = (uint8_t*)z + (at + lane * NV) * (BYTES / NV);
        if constexpr (BYTES == 4) *(uint32_t*)p = w[0];
        else if constexpr (BYTES == 8) *(uint2*)p = make_uint2(w[0], w[1]);
        else
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                *(uint4*)(p + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = lane * NV + j;
            if (e >= E) continue;
            if constexpr (SRC == MXQ_SRC_BF16) ((uint16_t*)z)[at + e] = to_bf(v[j]);
            else ((float*)z)[at + e] = v[j];
        }
    }
}

template <int NV, int SRC, bool VEC>
__global__ void __launch_bounds__(256) k_topk(const void* __restrict__ z, int64_t T, int E, int64_t ld, int k,
                                              int renorm, int32_t* __restrict__ ids, float* __restrict__ w) {
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    uint32_t key[NV];
    float v[NV];
    load_run<NV, SRC, VEC>(z, t * ld, E, lane, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = lane * NV + j < E ? order_key(v[j]) : 0u;
    float top = 0.0f, all = 0.0f;     // the largest logit; the sum over all experts
    float mine = 0.0f;                // lane j keeps the j-th pick
    int mine_id = 0;
    for (int p = 0; p < k; ++p) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j] > best) { best = key[j]; at = j; }
        const uint32_t m = wave_max(best);
        const int win = __builtin_ctzll(__ballot(best == m));
        const int id = __builtin_amdgcn_readlane(lane * NV + at, win);
        const float pick = key_value(m);
        if (p == 0) {
            top = pick;
            if (!renorm) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (key[j]) all += expf(v[j] - top);
                all = wave_sum(all);
            }
        }
        if (lane == p) { mine = pick; mine_id = id; }
        if (lane == win) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j == at) key[j] = 0u;
        }
    }
    mine = expf(mine - top);
    const float sum = renorm ? wave_sum(lane < k ? mine : 0.0f) : all;
    if (lane < k) {
        ids[t * k + lane] = mine_id;
        w[t * k + lane] = mine / sum;
    }
}

// dlogits_e = p_e (g_e - sum_c p_c g_c).  The wave holds the row as above and
// the picks one per lane.
template <int NV, int SRC, bool VEC>
__global__ void __launch_bounds__(256) k_topk_back(const void* __restrict__ z, int64_t T, int E, int64_t ld,
                                                   const int32_t* __restrict__ ids, int k, int renorm,
                                                   const float* __restrict__ dw, void* __restrict__ dz, int64_t ld_d) {
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    const int id = lane < k ? ids[t * k + lane] : -1;
    const float gk = lane < k ? dw[t * k + lane] : 0.0f;
    float v[NV], g[NV];
    bool in[NV];
    load_run<NV, SRC, VEC>(z, t * ld, E, lane, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = lane * NV + j < E;
        g[j] = 0.0f;
    }
    uint32_t chosen = 0u;
    for (int p = 0; p < k; ++p) {
        const int e = __builtin_amdgcn_readlane(id, p);
        const float ge = lane_value(gk, p);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (e == lane * NV + j && in[j]) { g[j] += ge; chosen |= 1u << j; }
    }
    if (renorm) {
#pragma unroll
        for (int j = 0; j < NV; ++j) in[j] = in[j] && (chosen >> j & 1u);
    }
    uint32_t top = 0u;  // the largest logit's key; a NaN's is above all
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (in[j]) top = max_u(top, order_key(v[j]));
    const float m = key_value(wave_max(top));
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        v[j] = in[j] ? expf(v[j] - m) : 0.0f;
        s += v[j];
    }
    s = wave_sum(s);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (in[j]) v[j] /= s;
        dot = fmaf(v[j], g[j], dot);
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = in[j] ? v[j] * (g[j] - dot) : 0.0f;
    store_run<NV, SRC, VEC>(dz, t * ld_d, E, lane, v);
}

// ---------------------------------------------------------------------------
// Stable counting sort of the assignments by expert.  A block owns a chunk of
// consecutive assignments and its 8 waves consecutive parts of it.  Within a
// wave, lanes of equal expert find each other by one ballot per bit of the
// expert, so ranks follow the order of the assignments without a serial
// step.  More than one chunk: k_sort_count leaves every chunk's counts in the
// workspace first, and every block of k_sort_place adds up the chunks before
// its own.
// ---------------------------------------------------------------------------
constexpr int SORT_NT = 512, SORT_W = SORT_NT / 64;
// Up to SORT_ONE assignments one block is faster than two launches; above, at
// most SORT_BLOCKS chunks, since every block reads all chunks' counts.
constexpr int64_t SORT_ONE = 4096, SORT_CHUNK = 1024, SORT_BLOCKS = 256;

inline int64_t sort_chunk(int64_t n) {
    if (n <= SORT_ONE) return SORT_ONE;
    const int64_t c = (n + SORT_BLOCKS - 1) / SORT_BLOCKS;
    return c <= SORT_CHUNK ? SORT_CHUNK : (c + SORT_NT - 1) / SORT_NT * SORT_NT;
}

// Inclusive sums over the block's threads; `sums` holds SORT_W values.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* sums) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t x = __shfl_up(v, d, 64);
        v += lane >= d ? x : 0;
    }
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += sums[w];
    return v;
}

__global__ void __launch_bounds__(SORT_NT) k_sort_count(const int32_t* __restrict__ ids, int64_t n, int64_t chunk,
                                                        int G, int32_t* __restrict__ counts) {
    extern __shared__ int32_t cnt[];
    for (int g = threadIdx.x; g < G; g += SORT_NT) cnt[g] = 0;
    __syncthreads();
    const int64_t a = (int64_t)blockIdx.x * chunk, b = a + chunk < n ? a + chunk : n;
    for (int64_t i = a + threadIdx.x; i < b; i += SORT_NT) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)G) atomicAdd(&cnt[e], 1);  // whole numbers: any order gives the same counts
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += SORT_NT) counts[(int64_t)blockIdx.x * G + g] = cnt[g];
}

// counts == nullptr: the only chunk.
__global__ void __launch_bounds__(SORT_NT) k_sort_place(const int32_t* __restrict__ ids, int64_t n, int64_t chunk,
                                                        int nchunks, int G, int k,
                                                        const int32_t* __restrict__ counts, int64_t* __restrict__ off,
                                                        int32_t* __restrict__ src, int32_t* __restrict__ pos) {
    extern __shared__ int32_t cnt[];  // [SORT_W][G]: each wave's counts, then its next row per expert
    __shared__ int32_t sums[SORT_W], all_of[SORT_NT], before_of[SORT_NT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < SORT_W * G; i += SORT_NT) cnt[i] = 0;
    __syncthreads();
    const int64_t a = (int64_t)blockIdx.x * chunk, b = a + chunk < n ? a + chunk : n;
    const int64_t part = chunk / SORT_W;
    const int64_t wa = a + wave * part < b ? a + wave * part : b, wb = wa + part < b ? wa + part : b;
    int32_t* mine = cnt + wave * G;
    for (int64_t i = wa + lane; i < wb; i += 64) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)G) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // counts of the other chunks: for up to SORT_NT experts P threads share one
    const int P = counts && G <= SORT_NT ? SORT_NT / G : 0;
    if (P) {
        int32_t x_all = 0, x_before = 0;
        const int g = tid % G, p = tid / G;
        if (p < P) {
#pragma unroll 8
            for (int c = p; c < nchunks; c += P) {
                const int32_t x = counts[(int64_t)c * G + g];
                x_all += x;
                x_before += c < (int)blockIdx.x ? x : 0;
            }
        }
        all_of[tid] = x_all;
        before_of[tid] = x_before;
        __syncthreads();
    }
    // thread i has the run of G / SORT_NT experts from per * i
    const int per = (G + SORT_NT - 1) / SORT_NT, g0 = tid * per, g1 = g0 + per < G ? g0 + per : G;
    int32_t total = 0;
    for (int g = g0; g < g1; ++g) {
        int32_t before = 0, in_all = 0;
        if (P) {
            for (int p = 0; p < P; ++p) { in_all += all_of[p * G + g]; before += before_of[p * G + g]; }
        } else if (counts) {
#pragma unroll 8
            for (int c = 0; c < nchunks; ++c) {
                const int32_t x = counts[(int64_t)c * G + g];
                in_all += x;
                before += c < (int)blockIdx.x ? x : 0;
            }
        }
        int32_t run = total + before;  // what precedes in this run of experts, and in the chunks before
        for (int w = 0; w < SORT_W; ++w) {
            const int32_t x = cnt[w * G + g];
            cnt[w * G + g] = run;
            run += x;
        }
        total += counts ? in_all : run - total;
        if (blockIdx.x == 0) off[g + 1] = total;  // completed below
    }
    const int32_t upto = block_scan(total, sums);
    const int32_t base = upto - total;
    int32_t placed = 0;
    for (int w = 0; w < SORT_W; ++w) placed += sums[w];
    for (int g = g0; g < g1; ++g) {
        for (int w = 0; w < SORT_W; ++w) cnt[w * G + g] += base;
        if (blockIdx.x == 0) off[g + 1] += base;
    }
    if (blockIdx.x == 0 && tid == 0) off[0] = 0;
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < G) ++bits;
    for (int64_t i0 = wa; i0 < wb; i0 += 64) {
        const int64_t i = i0 + lane;
        const int e = i < wb ? ids[i] : -1;
        const bool ok = (unsigned)e < (unsigned)G;
        uint64_t same = __ballot(ok);
        for (int t = 0; t < bits; ++t) {
            const uint64_t one = __ballot((e >> t) & 1);
            same &= ((e >> t) & 1) ? one : ~one;
        }
        int32_t row = -1;
        if (ok) row = mine[e] + __builtin_popcountll(same & ((1ull << lane) - 1));
        __builtin_amdgcn_wave_barrier();
        if (ok && (same >> lane) == 1ull) mine[e] = row + 1;  // the last lane of its expert
        __builtin_amdgcn_wave_barrier();
        if (i < wb) {
            pos[i] = row;
            if (ok && src) src[row] = (int32_t)(i / k);
        }
    }
    if (src)
        for (int64_t r = (a > placed ? a : placed) + tid; r < b; r += SORT_NT) src[r] = -1;
}

// ---------------------------------------------------------------------------
// Token rows to their experts' rows, MX quantized.  A lane holds 16 values
// (half an MX block) of one token and writes their codes to every row that
// pos names: each token's row is read and quantized once, however many
// experts it goes to, and not at all if it goes to none.
// ---------------------------------------------------------------------------
template <int F, int SRC>
__global__ void __launch_bounds__(256) k_dispatch(const uint8_t* __restrict__ x, uint32_t n, uint32_t upr, int64_t ld,
                                                  const int32_t* __restrict__ pos, int k, int64_t R,
                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;  // n is even: both lanes of a block leave together
    const uint32_t t = i / upr, u = i - t * upr;
    const int32_t* p = pos + (int64_t)t * k;
    bool any = false;
    for (int j = 0; j < k; ++j) any = any || (uint64_t)(int64_t)p[j] < (uint64_t)R;
    if (!any) return;
    uint32_t v[16];
    if constexpr (SRC == MXQ_SRC_BF16) {
        const uint8_t* b = x + (int64_t)t * ld + (int64_t)u * 32;
        const uint4 c0 = ld_nt16(b), c1 = ld_nt16(b + 16);
        const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) { v[2 * j] = w[j] << 16; v[2 * j + 1] = w[j] & 0xFFFF0000u; }
    } else {
        const uint8_t* b = x + (int64_t)t * ld + (int64_t)u * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 c = ld_nt16(b + 16 * j);
            v[4 * j] = c.x; v[4 * j + 1] = c.y; v[4 * j + 2] = c.z; v[4 * j + 3] = c.w;
        }
    }
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j) { const uint32_t a = v[j] & 0x7FFFFFFFu; m = a > m ? a : m; }
    const uint32_t o = (uint32_t)__shfl_xor((int)m, 1, 64);
    m = o > m ? o : m;
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    uint8_t sb;
    if constexpr (F != E2M1) {
        const uint32_t lo8[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
        const uint32_t hi8[8] = {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]};
        mx_codes_row8<F>(lo8, m, codes.x, codes.y, sb);
        mx_codes_row8<F>(hi8, m, codes.z, codes.w, sb);
    } else {
        const bool bad = m >= 0x7F800000u;
        const int e = block_exp<E2M1>(m >> 23);
        const float sc = exp2i(e);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t* y = v + 8 * h;
            uint32_t r = cvt2_f32_fp4<0>(0u, as_float(y[0]), as_float(y[1]), sc);
            r = cvt2_f32_fp4<1>(r, as_float(y[2]), as_float(y[3]), sc);
            r = cvt2_f32_fp4<2>(r, as_float(y[4]), as_float(y[5]), sc);
            w[h] = cvt2_f32_fp4<3>(r, as_float(y[6]), as_float(y[7]), sc);
        }
        codes.x = bad ? 0u : w[0];
        codes.y = bad ? 0u : w[1];
        sb = bad ? (uint8_t)0xFF : (uint8_t)(e + 127);
    }
    for (int j = 0; j < k; ++j) {
        const int64_t r = p[j];
        if ((uint64_t)r >= (uint64_t)R) continue;
        if constexpr (F != E2M1) st_nt16(q + (r * upr + u) * 16, codes);
        else st_nt8(q + (r * upr + u) * 8, make_uint2(codes.x, codes.y));
        if (!(u & 1)) s[r * (upr >> 1) + (u >> 1)] = sb;
    }
}

// ---------------------------------------------------------------------------
// Expert rows back to their tokens, weighted.  A lane holds 16 bytes of one
// token's row.
// ---------------------------------------------------------------------------
template <int SRC> struct Vec {  // 16 bytes as binary32 values
    static constexpr int N = SRC == MXQ_SRC_BF16 ? 8 : 4;
    float f[N];
    __device__ __forceinline__ void set(const uint4 v) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (N == 8) { f[2 * j] = as_float(u[j] << 16); f[2 * j + 1] = as_float(u[j] & 0xFFFF0000u); }
            else f[j] = as_float(u[j]);
        }
    }
    __device__ __forceinline__ uint4 get() const {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (N == 8) u[j] = (uint32_t)to_bf(f[2 * j]) | (uint32_t)to_bf(f[2 * j + 1]) << 16;
            else u[j] = as_uint(f[j]);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <int SRC, int CU>
__global__ void __launch_bounds__(256) k_combine(const uint8_t* __restrict__ x, int64_t R, int64_t ld_x,
                                                 const int32_t* __restrict__ pos, uint32_t n, uint32_t upr, int k,
                                                 const float* __restrict__ w, uint8_t* __restrict__ y, int64_t ld_y) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;
    const uint32_t t = i / upr, u = i - t * upr;
    Vec<SRC> acc;
    acc.set(make_uint4(0u, 0u, 0u, 0u));
    const int32_t* p = pos + (int64_t)t * k;
    const float* wt = w ? w + (int64_t)t * k : nullptr;
    for (int j0 = 0; j0 < k; j0 += CU) {  // CU rows' loads at once
        uint4 raw[CU];
        float c[CU];
        bool ok[CU];
#pragma unroll
        for (int j = 0; j < CU; ++j) {
            const int64_t r = j0 + j < k ? p[j0 + j] : -1;
            ok[j] = (uint64_t)r < (uint64_t)R;
            c[j] = wt && ok[j] ? wt[j0 + j] : 1.0f;
            raw[j] = ok[j] ? ld_nt16(x + r * ld_x + (int64_t)u * 16) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < CU; ++j) {
            Vec<SRC> row;
            row.set(raw[j]);
            if (ok[j])
#pragma unroll
                for (int e = 0; e < Vec<SRC>::N; ++e) acc.f[e] = fmaf(c[j], row.f[e], acc.f[e]);
        }
    }
    st_nt16(y + (int64_t)t * ld_y + (int64_t)u * 16, acc.get());
}

// One block per token: dy's row in registers a slab at a time, against each
// of its expert rows in turn.
constexpr int CB_NT = 256, CB_NU = 4;
template <int SRC>
__global__ void __launch_bounds__(CB_NT) k_combine_back(const uint8_t* __restrict__ dy, int64_t ld_dy,
                                                        const int32_t* __restrict__ pos, int upr, int k,
                                                        const float* __restrict__ w, const uint8_t* __restrict__ x,
                                                        int64_t ld_x, int64_t R, uint8_t* __restrict__ dx,
                                                        int64_t ld_dx, float* __restrict__ dw) {
    __shared__ float part[64][CB_NT / 64];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (dw && (int)threadIdx.x < k)
        for (int i = 0; i < CB_NT / 64; ++i) part[threadIdx.x][i] = 0.0f;
    __syncthreads();
    for (int u0 = 0; u0 < upr; u0 += CB_NT * CB_NU) {
        Vec<SRC> d[CB_NU];
#pragma unroll
        for (int i = 0; i < CB_NU; ++i) {
            const int u = u0 + i * CB_NT + threadIdx.x;
            d[i].set(u < upr ? ld_nt16(dy + t * ld_dy + (int64_t)u * 16) : make_uint4(0u, 0u, 0u, 0u));
        }
        for (int j = 0; j < k; ++j) {
            const int64_t r = pos[t * k + j];
            if ((uint64_t)r >= (uint64_t)R) continue;
            const float c = w ? w[t * k + j] : 1.0f;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < CB_NU; ++i) {
                const int u = u0 + i * CB_NT + threadIdx.x;
                if (u < upr) {
                    if (dw) {
                        Vec<SRC> v;
                        v.set(ld_nt16(x + r * ld_x + (int64_t)u * 16));
#pragma unroll
                        for (int e = 0; e < Vec<SRC>::N; ++e) s = fmaf(v.f[e], d[i].f[e], s);
                    }
                    if (dx) {
                        Vec<SRC> v;
#pragma unroll
                        for (int e = 0; e < Vec<SRC>::N; ++e) v.f[e] = c * d[i].f[e];
                        st_nt16(dx + r * ld_dx + (int64_t)u * 16, v.get());
                    }
                }
            }
            if (dw) {
                s = wave_sum(s);
                if (lane == 0) part[j][wave] += s;
            }
        }
    }
    if (!dw) return;
    __syncthreads();
    if ((int)threadIdx.x < k) {
        float s = 0.0f;
        for (int i = 0; i < CB_NT / 64; ++i) s += part[threadIdx.x][i];
        dw[t * k + threadIdx.x] = s;
    }
}

// Whether every row of NV-element runs can move as vectors.
template <int NV> bool runs_aligned(const void* p, int64_t ld, int64_t E, int esz) {
    const int64_t run = NV * esz < 16 ? NV * esz : 16;
    return E % NV == 0 && (uintptr_t)p % run == 0 && ld * esz % run == 0;
}
template <int NV, int SRC>
hipError_t topk_nv(const void* z, int64_t T, int E, int64_t ld, int k, int renorm, int32_t* ids, float* w,
                   hipStream_t st) {
    const unsigned nb = (unsigned)((T + 3) / 4);
    if (runs_aligned<NV>(z, ld, E, SRC == MXQ_SRC_BF16 ? 2 : 4))
        k_topk<NV, SRC, true><<<nb, 256, 0, st>>>(z, T, E, ld, k, renorm, ids, w);
    else
        k_topk<NV, SRC, false><<<nb, 256, 0, st>>>(z, T, E, ld, k, renorm, ids, w);
    return hipGetLastError();
}
template <int NV, int SRC>
hipError_t topk_back_nv(const void* z, int64_t T, int E, int64_t ld, const int32_t* ids, int k, int renorm,
                        const float* dw, void* dz, int64_t ld_d, hipStream_t st) {
    const unsigned nb = (unsigned)((T + 3) / 4);
    const int esz = SRC == MXQ_SRC_BF16 ? 2 : 4;
    if (runs_aligned<NV>(z, ld, E, esz) && runs_aligned<NV>(dz, ld_d, E, esz))
        k_topk_back<NV, SRC, true><<<nb, 256, 0, st>>>(z, T, E, ld, ids, k, renorm, dw, dz, ld_d);
    else
        k_topk_back<NV, SRC, false><<<nb, 256, 0, st>>>(z, T, E, ld, ids, k, renorm, dw, dz, ld_d);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_topk(const void* z, int src, int64_t T, int64_t E, int64_t ld, int k, int renorm, int32_t* ids,
                           float* w, hipStream_t st) {
    const int e = (int)E;
    const bool bf = src == MXQ_SRC_BF16;
#define MXQ_GO(NV) (bf ? topk_nv<NV, MXQ_SRC_BF16>(z, T, e, ld, k, renorm, ids, w, st) \
                       : topk_nv<NV, MXQ_SRC_F32>(z, T, e, ld, k, renorm, ids, w, st))
    return e <= 64 ? MXQ_GO(1) : e <= 128 ? MXQ_GO(2) : e <= 256 ? MXQ_GO(4) : e <= 512 ? MXQ_GO(8) : MXQ_GO(16);
#undef MXQ_GO
}

hipError_t launch_moe_topk_backward(const void* z, int src, int64_t T, int64_t E, int64_t ld, const int32_t* ids,
                                    int k, int renorm, const float* dw, void* dz, int64_t ld_d, hipStream_t st) {
    const int e = (int)E;
    const bool bf = src == MXQ_SRC_BF16;
#define MXQ_GO(NV) (bf ? topk_back_nv<NV, MXQ_SRC_BF16>(z, T, e, ld, ids, k, renorm, dw, dz, ld_d, st) \
                       : topk_back_nv<NV, MXQ_SRC_F32>(z, T, e, ld, ids, k, renorm, dw, dz, ld_d, st))
    return e <= 64 ? MXQ_GO(1) : e <= 128 ? MXQ_GO(2) : e <= 256 ? MXQ_GO(4) : e <= 512 ? MXQ_GO(8) : MXQ_GO(16);
#undef MXQ_GO
}

int64_t moe_sort_bytes(int64_t n, int64_t G) {
    const int64_t chunks = (n + sort_chunk(n) - 1) / sort_chunk(n);
    return chunks > 1 ? chunks * G * 4 : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int k, int G, int64_t* off, int32_t* src, int32_t* pos,
                           void* ws, hipStream_t st) {
    const int64_t chunk = sort_chunk(n);
    const int nb = n ? (int)((n + chunk - 1) / chunk) : 1;
    int32_t* counts = nb > 1 ? (int32_t*)ws : nullptr;
    const size_t lds = (size_t)SORT_W * G * 4;
    if (lds > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)k_sort_place, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)lds);
        if (e != hipSuccess) return e;
    }
    if (counts) k_sort_count<<<nb, SORT_NT, (size_t)G * 4, st>>>(ids, n, chunk, G, counts);
    k_sort_place<<<nb, SORT_NT, lds, st>>>(ids, n, chunk, nb, G, k, counts, off, src, pos);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch_mx(const void* x, int src, int64_t T, int64_t C, int64_t ld, const int32_t* pos, int k,
                                  int fmt, int64_t R, uint8_t* q, uint8_t* s, hipStream_t st) {
    const uint32_t upr = (uint32_t)(C / 16), n = (uint32_t)(T * (C / 16));
    const unsigned nb = (n + 255u) / 256u;
    const uint8_t* b = (const uint8_t*)x;
#define MXQ_GO(F, S, ESZ) k_dispatch<F, S><<<nb, 256, 0, st>>>(b, n, upr, ld * ESZ, pos, k, R, q, s)
    if (src == MXQ_SRC_BF16) {
        if (fmt == E4M3) MXQ_GO(E4M3, MXQ_SRC_BF16, 2);
        else if (fmt == E5M2) MXQ_GO(E5M2, MXQ_SRC_BF16, 2);
        else MXQ_GO(E2M1, MXQ_SRC_BF16, 2);
    } else {
        if (fmt == E4M3) MXQ_GO(E4M3, MXQ_SRC_F32, 4);
        else if (fmt == E5M2) MXQ_GO(E5M2, MXQ_SRC_F32, 4);
        else MXQ_GO(E2M1, MXQ_SRC_F32, 4);
    }
#undef MXQ_GO
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void* x, int src, int64_t R, int64_t C, int64_t ld_x, const int32_t* pos,
                              int64_t T, int k, const float* w, void* y, int64_t ld_y, hipStream_t st) {
    const int esz = src == MXQ_SRC_BF16 ? 2 : 4;
    const uint32_t upr = (uint32_t)(C * esz / 16), n = (uint32_t)(T * upr);
    const unsigned nb = (n + 255u) / 256u;
#define MXQ_GO(S, CU) k_combine<S, CU><<<nb, 256, 0, st>>>((const uint8_t*)x, R, ld_x * esz, pos, n, upr, k, w, (uint8_t*)y, ld_y * esz)
    if (src == MXQ_SRC_BF16) {
        if (k <= 2) MXQ_GO(MXQ_SRC_BF16, 2);
        else if (k <= 4) MXQ_GO(MXQ_SRC_BF16, 4);
        else MXQ_GO(MXQ_SRC_BF16, 8);
    } else {
        if (k <= 2) MXQ_GO(MXQ_SRC_F32, 2);
        else if (k <= 4) MXQ_GO(MXQ_SRC_F32, 4);
        else MXQ_GO(MXQ_SRC_F32, 8);
    }
#undef MXQ_GO
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* dy, int src, int64_t T, int64_t C, int64_t ld_dy,
                                       const int32_t* pos, int k, const float* w, const void* x, int64_t ld_x,
                                       int64_t R, void* dx, int64_t ld_dx, float* dw, hipStream_t st) {
    const int esz = src == MXQ_SRC_BF16 ? 2 : 4;
    const int upr = (int)(C * esz / 16);
    if (src == MXQ_SRC_BF16)
        k_combine_back<MXQ_SRC_BF16><<<(unsigned)T, CB_NT, 0, st>>>((const uint8_t*)dy, ld_dy * esz, pos, upr, k, w,
                                                                   (const uint8_t*)x, ld_x * esz, R, (uint8_t*)dx,
                                                                   ld_dx * esz, dw);
    else
        k_combine_back<MXQ_SRC_F32><<<(unsigned)T, CB_NT, 0, st>>>((const uint8_t*)dy, ld_dy * esz, pos, upr, k, w,
                                                                  (const uint8_t*)x, ld_x * esz, R, (uint8_t*)dx,
                                                                  ld_dx * esz, dw);
    return hipGetLastError();
}

}  // namespace mxq
