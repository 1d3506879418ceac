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

// What the wave's lanes wrote to LDS is there for its other lanes: LDS keeps a
// wave's order, the compiler is told to.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int SRC> __device__ __forceinline__ float load_el(const void* p, int64_t i) {
    if constexpr (SRC == MXQ_SRC_BF16) return as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    else return ((const float*)p)[i];
}
__device__ __forceinline__ uint16_t to_bf(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// e^d for d <= 0 (NaN and -inf included): relative to the result the product's
// rounding is off by at most |d| 2^-24, the rounded log2 e by 0.22 of that (its
// own relative error is 1.3e-8), exp2 by one ulp.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504f); }

// ---------------------------------------------------------------------------
// Router.  One wave per token; lane l holds experts l * NV .. l * NV + NV - 1,
// so that among equal logits the lowest lane, and in it the lowest slot, is
// the lowest expert.  A pick is one maximum over the lanes' largest keys.
// Bound by its instructions (about 300 a wave, eight waves per SIMD): 8192
// tokens x 256 experts, top-8, 7.0 us (0.7 us of bytes); its gradient, 5.3 us
// for 16.8 MB, is near the bytes (2.7 us and the launch).
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
    int idx[NV];
    float v[NV];
    load_run<NV, SRC, VEC>(z, t * ld, E, lane, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        key[j] = lane * NV + j < E ? order_key(v[j]) : 0u;
        idx[j] = lane * NV + j;
    }
    // The lane's run in descending order, equal keys in the order of experts:
    // passes over the even and the odd pairs in turn, rolled.  (Every pass
    // unrolled, 1024 experts took 73 us for 16 tokens and 347 for 8192, against
    // 5.6 and 19.5; 512 experts 9.7 and 32, against 4.0 and 9.5.)
    auto order = [&](int j) __attribute__((always_inline)) {  // j - 1 and j
        const bool up = key[j] > key[j - 1];
        const uint32_t a = up ? key[j] : key[j - 1], b = up ? key[j - 1] : key[j];
        const int c = up ? idx[j] : idx[j - 1], d = up ? idx[j - 1] : idx[j];
        key[j - 1] = a; key[j] = b;
        idx[j - 1] = c; idx[j] = d;
    };
#pragma clang loop unroll(disable)
    for (int p = 0; p < NV / 2; ++p) {
#pragma unroll
        for (int j = 1; j < NV; j += 2) order(j);
#pragma unroll
        for (int j = 2; j < NV; j += 2) order(j);
    }
    const float top = key_value(wave_max(key[0]));
    float sum = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int j = 0; j < NV; ++j) sum += lane * NV + j < E ? exp_of(v[j] - top) : 0.0f;
        sum = wave_sum(sum);
    }
    float mine = 0.0f;  // lane j keeps the j-th pick
    int mine_id = 0;
    for (int p = 0; p < k; ++p) {
        const uint32_t m = wave_max(key[0]);
        const int win = __builtin_ctzll(__ballot(key[0] == m));
        const int id = __builtin_amdgcn_readlane(idx[0], win);
        if (lane == p) { mine = key_value(m); mine_id = id; }
        if (lane == win) {
#pragma unroll
            for (int j = 0; j < NV - 1; ++j) { key[j] = key[j + 1]; idx[j] = idx[j + 1]; }
            key[NV - 1] = 0u;
        }
    }
    mine = exp_of(mine - top);
    if (renorm) sum = wave_sum(lane < k ? mine : 0.0f);
    if (lane < k) {
        ids[t * k + lane] = mine_id;
        w[t * k + lane] = mine / sum;
    }
}

// dlogits_e = p_e (g_e - sum_c p_c g_c).  The picks are scattered over the row
// in LDS (as g, or renormalized as the finished values, which need the picks'
// logits only), the rest of the row is one pass in registers.
template <int NV, int SRC, bool VEC>
__global__ void __launch_bounds__(256) k_topk_back(const void* __restrict__ z, int64_t T, int E, int64_t ld,
                                                   const int32_t* __restrict__ ids, int k, int renorm,
                                                   const float* __restrict__ dw, void* __restrict__ dz, int64_t ld_d) {
    __shared__ float rows[4][64 * NV];
    float* row = rows[threadIdx.x >> 6];  // this wave's own: no barrier, LDS keeps a wave's order
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    const int id = lane < k ? ids[t * k + lane] : -1;
    const bool mine = (unsigned)id < (unsigned)E;
    const float gk = lane < k ? dw[t * k + lane] : 0.0f;
    float v[NV];
    if (!renorm) load_run<NV, SRC, VEC>(z, t * ld, E, lane, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) row[lane * NV + j] = 0.0f;
    wave_sync();
    if (renorm) {
        const float zk = mine ? load_el<SRC>(z, t * ld + id) : 0.0f;
        const float m = key_value(wave_max(mine ? order_key(zk) : 0u));
        float p = mine ? exp_of(zk - m) : 0.0f;
        const float s = wave_sum(p);
        p = mine ? p / s : 0.0f;
        const float dot = wave_sum(mine ? p * gk : 0.0f);
        if (mine) row[id] = p * (gk - dot);
    } else if (mine) {
        row[id] = gk;
    }
    wave_sync();
    float g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) g[j] = row[lane * NV + j];
    if (!renorm) {
        uint32_t top = 0u;  // the largest logit's key; a NaN's is above all
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane * NV + j < E) top = max_u(top, order_key(v[j]));
        const float m = key_value(wave_max(top));
        float s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = lane * NV + j < E ? exp_of(v[j] - m) : 0.0f;
            s += v[j];
            dot = fmaf(v[j], g[j], dot);
        }
        const float inv = 1.0f / wave_sum(s);
        dot = wave_sum(dot) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) g[j] = v[j] * inv * (g[j] - dot);
    }
    store_run<NV, SRC, VEC>(dz, t * ld_d, E, lane, g);
}

// ---------------------------------------------------------------------------
// Stable counting sort of the assignments by expert.  A block owns a chunk of
// consecutive assignments and its waves consecutive parts of it.  Within a wave,
// lanes of equal expert find each other by one ballot per bit of the expert, so
// ranks follow the order of the assignments without a serial step.  More than
// one chunk: k_sort_count leaves every chunk's counts in the workspace first, and
// every block of k_sort_place adds up the chunks before its own, unless there
// are many (k_sort_scan).  Bound by latency: 65536 assignments to 256 experts 2.6
// + 7.2 us, 480 in one block 4.6 us (6.9 with its waves filled one after another).
// ---------------------------------------------------------------------------
// Loops are kept rolled: a launch this short waits for its instructions more
// than it gains from unrolling (10 us unrolled against 7).
constexpr int SORT_NT = 1024;  // half as many beyond 1024 experts, whose counts per wave fill the LDS
// Up to SORT_LONG assignments one block is faster than two launches.  Above,
// short chunks put more CUs to work, but every block reads chunks' counts, so the
// chunks grow once there are more than 256.
constexpr int64_t SORT_SHORT = 1024, SORT_LONG = 4096;

inline int64_t sort_chunk(int64_t n) { return n > SORT_LONG && n <= 256 * SORT_SHORT ? SORT_SHORT : SORT_LONG; }
// Whether the chunks' counts are added up once, by a launch of its own (2.5 us),
// rather than by every block: beyond 64 chunks a thread, or where the experts
// outnumber the threads.  Measured, without / with: 131072 assignments to 1024
// experts 20.5 / 17.3 us, 65536 to 1024 15.4 / 16.2; 65536 to 2048 66 / 18; 2^23
// to 256 341 / 92; 2^23 to 8 82 / 67; 2^20 to 8 14.7 / 16.8.
inline bool sort_scans(int64_t chunks, int64_t G) {
    return chunks > 1 && (G > SORT_NT || chunks * G > 65536 || chunks > 256);
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

// The counts of many chunks into each expert's rows before the chunk, and in
// one row more all of its rows.  A block has 8 experts; a thread runs over a
// 128th of the chunks of one of them, twice.
constexpr int SCAN_G = 8, SCAN_S = 128;
__global__ void __launch_bounds__(SCAN_G * SCAN_S) k_sort_scan(int32_t* __restrict__ counts, int nchunks, int G) {
    __shared__ int32_t sums[SCAN_S][SCAN_G];
    const int j = threadIdx.x % SCAN_G, s = threadIdx.x / SCAN_G, g = (int)blockIdx.x * SCAN_G + j;
    const int len = (nchunks + SCAN_S - 1) / SCAN_S;
    const int c0 = s * len < nchunks ? s * len : nchunks, c1 = c0 + len < nchunks ? c0 + len : nchunks;
    int32_t sum = 0;
    if (g < G)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += counts[(int64_t)c * G + g];
    sums[s][j] = sum;
    __syncthreads();
    int32_t before = 0;
    for (int i = 0; i < s; ++i) before += sums[i][j];
    if (g >= G) return;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        const int32_t x = counts[(int64_t)c * G + g];
        counts[(int64_t)c * G + g] = before;
        before += x;
    }
    if (s == SCAN_S - 1) counts[(int64_t)nchunks * G + g] = before;
}

// counts == nullptr: the only chunk; scanned: k_sort_scan has been over them.  LDS: W = blockDim / 64 rows of G counts
// (each wave's, then its next row per expert), then the chunk's ids.
__global__ void __launch_bounds__(SORT_NT) k_sort_place(const int32_t* __restrict__ ids, int64_t n, int chunk,
                                                        int nchunks, int scanned, int G, int k,
                                                        const int32_t* __restrict__ counts, int64_t* __restrict__ off,
                                                        int32_t* __restrict__ src, int32_t* __restrict__ pos) {
    extern __shared__ int32_t cnt[];
    __shared__ int32_t sums[SORT_NT / 64], all_of[SORT_NT], before_of[SORT_NT];
    const int nt = blockDim.x, W = nt >> 6;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t a = (int64_t)blockIdx.x * chunk;
    const int size = (int)(n - a < chunk ? n - a : chunk);
    const int part = chunk / W, w0 = wave * part < size ? wave * part : size, w1 = w0 + part < size ? w0 + part : size;
    int32_t* mine = cnt + wave * G;
    int32_t* held = cnt + W * G;
    for (int i = lane; i < G; i += 64) mine[i] = 0;
    wave_sync();
    for (int i = w0 + lane; i < w1; i += 64) {
        const int e = ids[a + i];
        held[i] = e;
        if ((unsigned)e < (unsigned)G) atomicAdd(&mine[e], 1);
    }
    // counts of all chunks, and of those before: P threads share an expert
    const int P = counts && !scanned ? nt / G : 0;  // G <= nt
    if (P) {
        int32_t x_all = 0, x_before = 0;
        const int p = tid / G, g = tid - p * G;
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
    }
    __syncthreads();
    // thread i has the run of G / nt experts from per * i
    const int per = (G + nt - 1) / nt, g0 = tid * per, g1 = g0 + per < G ? g0 + per : G;
    auto counted = [&](int g, int32_t& before) __attribute__((always_inline)) {  // expert g's, and those of earlier chunks
        int32_t in_all = 0;
        before = 0;
        if (P) {
            for (int p = 0; p < P; ++p) { in_all += all_of[p * G + g]; before += before_of[p * G + g]; }
        } else if (scanned) {
            in_all = counts[(int64_t)nchunks * G + g];
            before = counts[(int64_t)blockIdx.x * G + g];
        } else {
#pragma unroll 8
            for (int w = 0; w < W; ++w) in_all += cnt[w * G + g];
        }
        return in_all;
    };
    int32_t total = 0, before = 0;
    for (int g = g0; g < g1; ++g) total += counted(g, before);
    int32_t base = total;  // sums over the threads
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t x = __shfl_up(base, d, 64);
        base += lane >= d ? x : 0;
    }
    if (lane == 63) sums[wave] = base;
    __syncthreads();
    base -= total;
    int32_t placed = 0;
    for (int w = 0; w < W; ++w) {
        base += w < wave ? sums[w] : 0;
        placed += sums[w];
    }
    for (int g = g0; g < g1; ++g) {
        const int32_t in_all = per == 1 ? total : counted(g, before);
        int32_t x[SORT_NT / 64], run = base + before;
#pragma unroll
        for (int w = 0; w < SORT_NT / 64; ++w) x[w] = w < W ? cnt[w * G + g] : 0;
#pragma unroll
        for (int w = 0; w < SORT_NT / 64; ++w) {
            if (w < W) cnt[w * G + g] = run;
            run += x[w];
        }
        base += in_all;
        if (blockIdx.x == 0) off[g + 1] = base;
    }
    if (blockIdx.x == 0 && tid == 0) off[0] = 0;
    __syncthreads();
    const int bits = 32 - __builtin_clz(G);  // enough for G - 1
    for (int i0 = w0; i0 < w1; i0 += 64) {
        const int i = i0 + lane;
        const int e = i < w1 ? held[i] : -1;
        const bool ok = (unsigned)e < (unsigned)G;
        uint64_t same = __ballot(ok);
        for (int t = 0; t < bits; ++t) {
            const uint64_t one = __ballot((e >> t) & 1);
            same &= ((e >> t) & 1) ? one : ~one;
        }
        int32_t row = -1;
        if (ok) row = mine[e] + __builtin_popcountll(same & ((1ull << lane) - 1));
        wave_sync();
        if (ok && (same >> lane) == 1ull) mine[e] = row + 1;  // the last lane of its expert
        wave_sync();
        if (i < w1) {
            pos[a + i] = row;
            if (ok && src) src[row] = (int32_t)((uint32_t)(a + i) / (uint32_t)k);
        }
    }
    if (src)
        for (int64_t r = (a > placed ? a : placed) + tid; r < a + size; r += nt) src[r] = -1;
}

// ---------------------------------------------------------------------------
// Token rows to their experts' rows, MX quantized.  A lane holds 16 values
// (half an MX block) of one token and writes their codes to every row that
// pos names: each token's row is read and quantized once, however many
// experts it goes to, and not at all if it goes to none.  Bound by HBM: 4096 x
// 4096 to eight places each (172 MB, four fifths of it written) 34 us.  Loads
// and stores are nontemporal: plain ones took 4% more on cold rows.
// ---------------------------------------------------------------------------
// WHOLE: rows of a multiple of 1024 columns and up to 64 places, so that a wave
// has one token: its places sit in one register across the lanes, only those
// inside the buffers are visited, and one store writes eight places' scales.
template <int F, int SRC, bool WHOLE>
__global__ void __launch_bounds__(256) k_dispatch(const uint8_t* __restrict__ x, uint32_t n, uint32_t upr, int64_t ld,
                                                  const int32_t* __restrict__ pos, int k, int64_t R,
                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;  // n is even: both lanes of a block leave together
    const uint32_t t = WHOLE ? __builtin_amdgcn_readfirstlane(i) / upr : i / upr, u = i - t * upr;
    const int32_t* p = pos + (int64_t)t * k;
    const int lane = threadIdx.x & 63;
    int32_t to[WHOLE ? 1 : 8];  // WHOLE: place `lane`; else the first eight, more are read again below
    uint64_t inside = 0;
    if constexpr (WHOLE) {
        to[0] = lane < k ? p[lane] : -1;
        inside = __ballot((uint64_t)(int64_t)to[0] < (uint64_t)R);
        if (!inside) return;
    } else {
        bool any = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            to[j] = j < k ? p[j] : -1;
            any = any || (uint64_t)(int64_t)to[j] < (uint64_t)R;
        }
        for (int j = 8; j < k; ++j) any = any || (uint64_t)(int64_t)p[j] < (uint64_t)R;
        if (!any) return;
    }
    constexpr bool PK = SRC == MXQ_SRC_BF16;  // two to a word
    uint32_t v[PK ? 8 : 16], m;
    {
        const uint8_t* b = x + (int64_t)t * ld + (int64_t)u * (PK ? 32 : 64);
#pragma unroll
        for (int j = 0; j < (PK ? 2 : 4); ++j) {
            const uint4 c = ld_nt16(b + 16 * j);
            v[4 * j] = c.x; v[4 * j + 1] = c.y; v[4 * j + 2] = c.z; v[4 * j + 3] = c.w;
        }
    }
    if constexpr (PK) {
        uint32_t w = v[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int j = 1; j < 8; ++j) w = pk_max_u16(w, v[j] & 0x7FFF7FFFu);
        m = max_u(w << 16, w & 0xFFFF0000u);
    } else {
        m = 0u;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max_u(m, v[j] & 0x7FFFFFFFu);
    }
    m = max_u(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));  // the pair's other lane
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    const bool bad = m >= 0x7F800000u;
    const int e = block_exp<F>(m >> 23);
    const float sc = exp2i(e);
    if constexpr (F == E2M1) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t* y = v + (PK ? 4 : 8) * h;
            if constexpr (PK) {
                w[h] = cvt2_bf16_fp4<0>(0u, y[0], sc);
                w[h] = cvt2_bf16_fp4<1>(w[h], y[1], sc);
                w[h] = cvt2_bf16_fp4<2>(w[h], y[2], sc);
                w[h] = cvt2_bf16_fp4<3>(w[h], y[3], sc);
            } else {
                w[h] = cvt2_f32_fp4<0>(0u, as_float(y[0]), as_float(y[1]), sc);
                w[h] = cvt2_f32_fp4<1>(w[h], as_float(y[2]), as_float(y[3]), sc);
                w[h] = cvt2_f32_fp4<2>(w[h], as_float(y[4]), as_float(y[5]), sc);
                w[h] = cvt2_f32_fp4<3>(w[h], as_float(y[6]), as_float(y[7]), sc);
            }
        }
        codes.x = bad ? 0u : w[0];
        codes.y = bad ? 0u : w[1];
    } else {
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if constexpr (PK) {
                const uint32_t lim = (uint32_t)(e + 127 + FmtInfo<F>::emax) << 7 | FmtInfo<F>::max_mant_bf16;
                const uint32_t lim2 = lim | (lim << 16);
                w[h] = cvt2_bf16_fp8<F>(0u, clamp2_bf16(v[2 * h], lim2), sc, false);
                w[h] = cvt2_bf16_fp8<F>(w[h], clamp2_bf16(v[2 * h + 1], lim2), sc, true);
            } else {
                const uint32_t lim = (uint32_t)(e + 127 + FmtInfo<F>::emax) << 23 | FmtInfo<F>::max_mant_f32;
                const uint32_t* y = v + 4 * h;
                w[h] = cvt2_f32_fp8<F>(0u, as_float(clamp_f32(y[0], lim)), as_float(clamp_f32(y[1], lim)), sc, false);
                w[h] = cvt2_f32_fp8<F>(w[h], as_float(clamp_f32(y[2], lim)), as_float(clamp_f32(y[3], lim)), sc, true);
            }
            if (bad) w[h] = 0x7F7F7F7Fu;
        }
        codes = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint8_t sb = bad ? (uint8_t)0xFF : (uint8_t)(e + 127);
    auto put = [&](int64_t r) __attribute__((always_inline)) {
        if constexpr (F != E2M1) st_nt16(q + (r * upr + u) * 16, codes);
        else st_nt8(q + (r * upr + u) * 8, make_uint2(codes.x, codes.y));
    };
    if constexpr (WHOLE) {
        for (uint64_t left = inside; left; left &= left - 1)
            put((uint32_t)__builtin_amdgcn_readlane(to[0], __builtin_ctzll(left)));
        // lane 8 j + d: the scales of the wave's blocks 4 d .. 4 d + 3, to place j
        uint32_t four = 0u;
#pragma unroll
        for (int b = 0; b < 4; ++b) four |= (uint32_t)__shfl((int)sb, 8 * (lane & 7) + 2 * b, 64) << (8 * b);
        const uint32_t at = (__builtin_amdgcn_readfirstlane(u) >> 1) + 4 * (lane & 7);
        for (int j = lane >> 3; j - (lane >> 3) < k; j += 8) {
            const int64_t r = __shfl(to[0], j, 64);
            if (j < k && (uint64_t)r < (uint64_t)R) *(uint32_t*)(s + r * (upr >> 1) + at) = four;
        }
    } else {
        auto put_one = [&](int32_t row) __attribute__((always_inline)) {
            if ((uint64_t)(int64_t)row >= (uint64_t)R) return;
            put(row);
            if (!(u & 1)) s[(int64_t)row * (upr >> 1) + (u >> 1)] = sb;
        };
#pragma unroll
        for (int j = 0; j < 8; ++j) put_one(to[j]);
        for (int j = 8; j < k; ++j) put_one(p[j]);
    }
}

// ---------------------------------------------------------------------------
// Expert rows back to their tokens, weighted.  A lane holds 16 bytes of one
// token's row and loads up to eight experts' pieces before it adds: 32768 rows
// of 7168 bf16 to 4096 tokens (529 MB) 86 us, 6.1 TB/s, the rate of a copy; one
// row's load at a time took 100 us.
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

// dy's row in registers, a slab of NTT NU vectors at a time, against the token's
// expert rows, JU at a time so that their loads overlap.  A wave takes a narrow
// row (4999 tokens of 128 bf16, seven places: 10.7 us, 18.7 with a block each),
// a block a wide one.  Few tokens: the places of each are cut over blocks (per
// at a time), whose sums do not meet (127 tokens of 7328 binary32, eight places:
// 18.7 us, 26.2 uncut).
// 24006 rows of 4096 bf16 (427 MB, half of it written) 80 us, 5.3 TB/s; plain
// loads and stores took 2-7% more on cold rows, three rows at a time the same.
constexpr int CB_NT = 256;
template <int SRC, int NU, int NTT, int JU>
__global__ void __launch_bounds__(CB_NT) k_combine_back(const uint8_t* __restrict__ dy, int64_t ld_dy,
                                                        const int32_t* __restrict__ pos, int64_t T, int upr, int k,
                                                        int per, const float* __restrict__ w,
                                                        const uint8_t* __restrict__ x, int64_t ld_x, int64_t R,
                                                        uint8_t* __restrict__ dx, int64_t ld_dx,
                                                        float* __restrict__ dw) {
    constexpr int TPB = CB_NT / NTT, NW = NTT / 64;
    __shared__ float parts[TPB][64][NW], scales[TPB][64];
    __shared__ int32_t places[TPB][64 + JU];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wid / NW, wave = wid % NW, lt = threadIdx.x % NTT;
    const int64_t t = (int64_t)blockIdx.x * TPB + slot;
    if (t >= T) return;  // a wave of its own, or (TPB == 1) not at all
    auto sync = [&] {
        if constexpr (NW == 1) wave_sync();
        else __syncthreads();
    };
    float (&part)[64][NW] = parts[slot];
    float* scale = scales[slot];
    int32_t* to = places[slot];
    const int ja = (int)blockIdx.y * per, n = k - ja < per ? k - ja : per;
    pos += t * k + ja;
    for (int j = lt; j < n + JU; j += NTT) {  // past the last: none
        const int32_t r = j < n ? pos[j] : -1;
        to[j] = (uint64_t)(int64_t)r < (uint64_t)R ? r : -1;
        if (j < n) {
            scale[j] = w ? w[t * k + ja + j] : 1.0f;
            for (int i = 0; i < NW; ++i) part[j][i] = 0.0f;
        }
    }
    sync();
    for (int u0 = lt; u0 - lt < upr; u0 += NTT * NU) {
        Vec<SRC> d[NU];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = u0 + i * NTT;
            d[i].set(u < upr ? ld_nt16(dy + t * ld_dy + (int64_t)u * 16) : make_uint4(0u, 0u, 0u, 0u));
        }
        for (int j0 = 0; j0 < n; j0 += JU) {
            int64_t r[JU];
            bool ok[JU];  // the same for the whole wave
            uint4 raw[JU][NU];
#pragma unroll
            for (int h = 0; h < JU; ++h) {
                r[h] = __builtin_amdgcn_readfirstlane(to[j0 + h]);
                ok[h] = r[h] >= 0;
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    const int u = u0 + i * NTT;
                    raw[h][i] = dw && ok[h] && u < upr ? ld_nt16(x + r[h] * ld_x + (int64_t)u * 16)
                                                      : make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (dx) {
#pragma unroll
                for (int h = 0; h < JU; ++h) {
                    const float c = ok[h] ? scale[j0 + h] : 0.0f;
#pragma unroll
                    for (int i = 0; i < NU; ++i) {
                        const int u = u0 + i * NTT;
                        Vec<SRC> v;
#pragma unroll
                        for (int e = 0; e < Vec<SRC>::N; ++e) v.f[e] = c * d[i].f[e];
                        if (ok[h] && u < upr) st_nt16(dx + r[h] * ld_dx + (int64_t)u * 16, v.get());
                    }
                }
            }
            if (dw) {
#pragma unroll
                for (int h = 0; h < JU; ++h) {
                    if (!ok[h]) continue;
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < NU; ++i) {
                        Vec<SRC> v;
                        v.set(raw[h][i]);
#pragma unroll
                        for (int e = 0; e < Vec<SRC>::N; ++e)
                            if (u0 + i * NTT < upr) s = fmaf(v.f[e], d[i].f[e], s);
                    }
                    s = wave_sum(s);
                    if (lane == 0) part[j0 + h][wave] += s;
                }
            }
        }
    }
    if (!dw) return;
    sync();
    if (lt < n) {
        float s = 0.0f;
        for (int i = 0; i < NW; ++i) s += part[lt][i];
        dw[t * k + ja + lt] = s;
    }
}

template <int SRC, int NU, int NTT, int JU>
hipError_t combine_back(const uint8_t* dy, int64_t ld_dy, const int32_t* pos, int64_t T, int upr, int k, const float* w,
                        const uint8_t* x, int64_t ld_x, int64_t R, uint8_t* dx, int64_t ld_dx, float* dw,
                        hipStream_t st) {
    constexpr int TPB = CB_NT / NTT;
    const int64_t nb = (T + TPB - 1) / TPB, most = LAUNCH_THREADS / CB_NT;
    const int groups = (k + JU - 1) / JU, cut = nb >= 1024 ? 1 : groups * nb <= 1024 ? groups : (int)(1024 / nb);
    const int per = (groups + cut - 1) / cut * JU;
    for (int64_t b0 = 0; b0 < nb; b0 += most) {
        const int64_t b = nb - b0 < most ? nb - b0 : most, t0 = b0 * TPB, at = t0 * k;
        k_combine_back<SRC, NU, NTT, JU><<<dim3((unsigned)b, (unsigned)((k + per - 1) / per)), CB_NT, 0, st>>>(
            dy + t0 * ld_dy, ld_dy, pos + at, T - t0, upr, k, per, w ? w + at : nullptr, x, ld_x, R, dx, ld_dx,
            dw ? dw + at : nullptr);
    }
    return hipGetLastError();
}

// Whether every row of NV-element runs can move as vectors.
template <int NV> bool runs_aligned(const void* p, int64_t ld, int64_t E, int esz) {
    const int64_t run = NV * esz < 16 ? NV * esz : 16;
    return E % NV == 0 && (uintptr_t)p % run == 0 && ld * esz % run == 0;
}
template <int NV, int SRC>
hipError_t topk_nv(const void* z, int64_t T, int E, int64_t ld, int k, int renorm, int32_t* ids, float* w,
                   hipStream_t st) {
    constexpr int esz = SRC == MXQ_SRC_BF16 ? 2 : 4;
    const bool vec = runs_aligned<NV>(z, ld, E, esz);
    for (int64_t t0 = 0; t0 < T; t0 += LAUNCH_THREADS / 64) {
        const int64_t n = T - t0 < LAUNCH_THREADS / 64 ? T - t0 : LAUNCH_THREADS / 64;
        const unsigned nb = (unsigned)((n + 3) / 4);
        const uint8_t* from = (const uint8_t*)z + t0 * ld * esz;
        if (vec) k_topk<NV, SRC, true><<<nb, 256, 0, st>>>(from, n, E, ld, k, renorm, ids + t0 * k, w + t0 * k);
        else k_topk<NV, SRC, false><<<nb, 256, 0, st>>>(from, n, E, ld, k, renorm, ids + t0 * k, w + t0 * k);
    }
    return hipGetLastError();
}
template <int NV, int SRC>
hipError_t topk_back_nv(const void* z, int64_t T, int E, int64_t ld, const int32_t* ids, int k, int renorm,
                        const float* dw, void* dz, int64_t ld_d, hipStream_t st) {
    constexpr int esz = SRC == MXQ_SRC_BF16 ? 2 : 4;
    const bool vec = runs_aligned<NV>(z, ld, E, esz) && runs_aligned<NV>(dz, ld_d, E, esz);
    for (int64_t t0 = 0; t0 < T; t0 += LAUNCH_THREADS / 64) {
        const int64_t n = T - t0 < LAUNCH_THREADS / 64 ? T - t0 : LAUNCH_THREADS / 64, at = t0 * k;
        const unsigned nb = (unsigned)((n + 3) / 4);
        const uint8_t* from = (const uint8_t*)z + t0 * ld * esz;
        uint8_t* to = (uint8_t*)dz + t0 * ld_d * esz;
        if (vec) k_topk_back<NV, SRC, true><<<nb, 256, 0, st>>>(from, n, E, ld, ids + at, k, renorm, dw + at, to, ld_d);
        else k_topk_back<NV, SRC, false><<<nb, 256, 0, st>>>(from, n, E, ld, ids + at, k, renorm, dw + at, to, ld_d);
    }
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

// Dynamic LDS of k_sort_place: its waves' counts and the chunk's ids.
constexpr size_t sort_lds(int nt, int G, int chunk) { return ((size_t)nt / 64 * G + chunk) * 4; }
constexpr size_t SORT_LDS = sort_lds(SORT_NT / 2, 4096, SORT_LONG);  // the most
static_assert(SORT_LDS >= sort_lds(SORT_NT, 1024, SORT_LONG), "the most");

int64_t moe_sort_bytes(int64_t n, int64_t G) {
    const int64_t chunks = (n + sort_chunk(n) - 1) / sort_chunk(n);
    return chunks > 1 ? (chunks + sort_scans(chunks, G)) * G * 4 : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int k, int G, int64_t* off, int32_t* src, int32_t* pos,
                           void* ws, hipStream_t st) {
    int chunk = (int)sort_chunk(n);
    const int nb = n ? (int)((n + chunk - 1) / chunk) : 1;
    int32_t* counts = nb > 1 ? (int32_t*)ws : nullptr;
    const int nt = G <= 1024 ? SORT_NT : SORT_NT / 2;
    if (nb == 1) chunk = (int)(n > nt ? (n + nt - 1) / nt * nt : nt);  // a lone block's waves share what there is evenly
    const size_t lds = sort_lds(nt, G, chunk);
    if (lds > 48 * 1024) {
        // the limit is the kernel's, not the launch's: always the same one, so that no other thread's call lowers it
        const hipError_t e = hipFuncSetAttribute((const void*)k_sort_place, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)SORT_LDS);
        if (e != hipSuccess) return e;
    }
    if (counts) k_sort_count<<<nb, SORT_NT, (size_t)G * 4, st>>>(ids, n, chunk, G, counts);
    const int scan = sort_scans(nb, G);
    if (scan) k_sort_scan<<<(unsigned)((G + SCAN_G - 1) / SCAN_G), SCAN_G * SCAN_S, 0, st>>>(counts, nb, G);
    k_sort_place<<<nb, nt, lds, st>>>(ids, n, chunk, nb, scan, G, k, counts, off, src, pos);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch_mx(const void* x, int src, int64_t T, int64_t C, int64_t ld, const int32_t* pos, int k,
                                  int fmt, int64_t R, uint8_t* q, uint8_t* s, hipStream_t st) {
    const uint32_t upr = (uint32_t)(C / 16), n = (uint32_t)(T * (C / 16));
    const unsigned nb = (n + 255u) / 256u;
    const uint8_t* b = (const uint8_t*)x;
    const bool whole = upr % 64 == 0 && k <= 64 && (uintptr_t)s % 4 == 0;
#define MXQ_GO(F, S, ESZ)                                                                                \
    (whole ? k_dispatch<F, S, true><<<nb, 256, 0, st>>>(b, n, upr, ld * ESZ, pos, k, R, q, s)            \
           : k_dispatch<F, S, false><<<nb, 256, 0, st>>>(b, n, upr, ld * ESZ, pos, k, R, q, s))
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
#define MXQ_GO(S, NU, NTT, JU)                                                                                      \
    combine_back<S, NU, NTT, JU>((const uint8_t*)dy, ld_dy * esz, pos, T, upr, k, w, (const uint8_t*)x, ld_x * esz, R, \
                                 (uint8_t*)dx, ld_dx * esz, dw, st)
#define MXQ_SIZES(S)                        \
    (upr <= 64    ? MXQ_GO(S, 1, 64, 4)     \
     : upr <= 128 ? MXQ_GO(S, 2, 64, 4)     \
     : upr <= 256 ? MXQ_GO(S, 1, CB_NT, 4)  \
     : upr <= 512 ? MXQ_GO(S, 2, CB_NT, 2)  \
                  : MXQ_GO(S, 4, CB_NT, 2))
    return src == MXQ_SRC_BF16 ? MXQ_SIZES(MXQ_SRC_BF16) : MXQ_SIZES(MXQ_SRC_F32);
#undef MXQ_SIZES
#undef MXQ_GO
}

}  // namespace mxq
