// route.cu -- the router of an expert layer on its own: topk experts and their
// gates from a [tokens, experts] score matrix (softmax or sigmoid scores, a
// bias that takes part in the choice only, groups of experts of which the best
// stay open, renormalised and scaled gates, tokens per expert), and the
// gradient of the gates with respect to the logits.
//
// One warp orders a row; lane l holds V consecutive experts of it.  The choice
// is k rounds of a warp-wide maximum; what decides it is an order in which ties
// go to the lower expert, so the result is a function of the row alone.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"

namespace kosmos {

namespace {

constexpr int ROUTE_WARPS = 8;
constexpr int ROUTE_THREADS = ROUTE_WARPS * 32;
constexpr uint32_t FULL = 0xFFFFFFFFu;
#ifndef MINB
#define MINB 3
#endif
#ifndef RRF
#define RRF 32
#endif
constexpr int ROUTE_ROWS_FROM = RRF;  // tokens per SM from which a warp takes several rows at a time

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *gate;
    int32_t *counts;
    uint32_t *ticket;   // workspace: blocks that have added their counts
    int32_t *acc;       // workspace: [E] counts so far, zero between calls
    int64_t T, ld;
    int E, k, G, GK, group_top, score, renorm;
    float scale;
    // set by the launcher
    bool vec;                         // runs of experts are loaded whole
    int hist_words, row_words;        // shared memory: counts, then a row of values per warp (groups only)
    int rows, slots;                  // rows a warp takes at a time, lanes that hold a row's choices
    bool lane_groups;                 // a group is a run of 1 << lp_log2 lanes
    int gs, gsp, gmul, lp_log2;       // group size, its stride in shared memory, division by gs, lanes per group
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Lane l holds the V consecutive experts from l * V on: the lowest of tied
// experts is then in the lowest lane, and a group is often a run of lanes.
template <int V> __device__ __forceinline__ int expert_of(int lane, int v) { return lane * V + v; }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
    return v;
}
template <typename F> __device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
    return v;
}
// The gates of the chosen experts (slots lanes per row; logit x, open or
// closed).  m, z: the row's maximum and sum of exponentials (softmax without
// renorm).  Ratios of p are taken relative to the largest chosen one, so that
// small scores keep their precision.
__device__ __forceinline__ float route_gate(const RouteParams &p, int slots, float x, bool open, float m, float z) {
    if (!p.renorm) {
        if (!open) return 0.f;
        return p.scale * (p.score == KOSMOS_SCORE_SOFTMAX ? expf(x - m) / z : 1.0f / (1.0f + expf(-x)));
    }
    float top = open ? x : -INFINITY;
    for (int d = slots / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
    float w = 0.f;
    if (open) {
        if (p.score == KOSMOS_SCORE_SOFTMAX) {
            w = expf(x - top);
        } else {
            top = fminf(top, 0.f);
            w = x > 0.f ? 1.0f / (1.0f + expf(-x)) : expf(x - top) / (1.0f + expf(x));
        }
    }
    float sum = w;
    for (int d = slots / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
    return open ? p.scale * (w / sum) : 0.f;
}

// ------------------------------------------------------------ fp32 choice
// How a kernel orders a row's experts: without a bias by their logits, which
// the scores rise with; else by s = p + bias in fp32.  Rows in which two
// neighbours in the order, or the groups either side of the border, are closer
// than the scores' rounding error are chosen again in 64 bits.
enum RouteMode : int { BY_LOGIT = 0, BY_SIGMOID = 1, BY_SOFTMAX = 2 };

// Order-preserving map of floats to unsigned integers (-0 as +0).  Closed
// experts have the key of -inf, and so have the places beyond E, which
// come last of all because ties go to the lower expert.
constexpr uint32_t KEY_NONE = 0u, KEY_CLOSED = 0x007FFFFFu;
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// A row's values, in loads of up to 16 bytes where rows and runs allow it.
// Beyond E: -inf.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *row, int E, int lane, bool vec, T *r) {
    constexpr int W = V * sizeof(T) < 16 ? V : 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int c = 0; c < V; c += W) {
        const int e0 = lane * V + c;
        if (vec) {
            if (e0 < E) {
                if constexpr (W * sizeof(T) == 16)
                    *reinterpret_cast<uint4 *>(r + c) = __ldg(reinterpret_cast<const uint4 *>(row + e0));
                else if constexpr (W * sizeof(T) == 8)
                    *reinterpret_cast<uint2 *>(r + c) = __ldg(reinterpret_cast<const uint2 *>(row + e0));
                else
                    *reinterpret_cast<uint32_t *>(r + c) = __ldg(reinterpret_cast<const uint32_t *>(row + e0));
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) r[c + i] = from_f32<T>(-INFINITY);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) r[c + i] = e0 + i < E ? row[e0 + i] : from_f32<T>(-INFINITY);
        }
    }
}

constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// p in fp32 (rz = 1 / z): x = -inf gives 0.
template <int MODE> __device__ __forceinline__ float fast_p(float x, float m, float rz) {
    if (MODE == BY_SIGMOID) return rcp(1.0f + ex2(-LOG2E * x));
    return ex2(LOG2E * (x - m)) * rz;
}

// Bounds on the distance between an fp32 score and the 64-bit one.  Sigmoid:
// the exponential is off by 2 + 1.2 |x| steps of 2^-23 (argument and result),
// which p (1 - p) brings under 6e-8; sum and reciprocal 3e-7 p; the bias'
// addition 6e-8 |s|.  Softmax: e^-y of a term y below the maximum is off by
// (2.5 + 1.7 y) steps, at most 3e-7 of the largest term; the row's sum and its
// reciprocal by 5e-6 (its terms' errors weigh at most ln 1024, and there are 37
// additions); the bias as above.
template <int MODE> __device__ __forceinline__ float score_error(float s, float p, float rz) {
    if (MODE == BY_LOGIT) return 0.f;
    return (MODE == BY_SIGMOID ? 5e-7f : 3e-7f * rz + 5e-6f * p) + 1.2e-7f * fabsf(s);
}

// (t1, t2): a lane's best two values; afterwards those of its 1 << n lanes.
__device__ __forceinline__ void join_top2(float &t1, float &t2, int n) {
    for (int d = 1; d < (1 << n); d <<= 1) {
        const float o1 = __shfl_xor_sync(FULL, t1, d), o2 = __shfl_xor_sync(FULL, t2, d);
        t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
        t1 = fmaxf(t1, o1);
    }
}

// Whether this lane's group, group lane >> lp_log2 with best values (t1, t2),
// stays open.  err > 0: the error of the values behind a group's score; near
// then tells that the border lies between scores that it does not separate.
__device__ __forceinline__ bool group_open(const RouteParams &p, float t1, float t2, int lane, float err, bool &near) {
    const int g = lane >> p.lp_log2;
    float ge = err + 2.4e-7f * fabsf(t1);  // two scores' errors and their sum's
    if (p.group_top == 2 && t2 != -INFINITY) {
        ge += 2.4e-7f * fabsf(t2);
        t1 += t2;
    }
    // a group's lanes share the comparison with the others
    int rank = 0;
    const int lp = 1 << p.lp_log2;
    for (int o0 = 0; o0 < p.G; o0 += lp) {
        const int o = o0 + (lane & (lp - 1));
        const float v = __shfl_sync(FULL, t1, o << p.lp_log2);
        rank += o < p.G && (v > t1 || (v == t1 && o < g)) ? 1 : 0;
    }
    for (int d = 1; d < lp; d <<= 1) rank += __shfl_xor_sync(FULL, rank, d);
    const bool in = g < p.G && rank < p.GK;
    if (err > 0.f) {
        // by keys: the least of the open groups' lower bounds and the largest of the others' upper bounds
        const uint32_t lo = __reduce_min_sync(FULL, in ? float_key(t1 - ge) : 0xFFFFFFFFu);
        const uint32_t hi = __reduce_max_sync(FULL, !in && g < p.G && t1 != -INFINITY ? float_key(t1 + ge) : KEY_NONE);
        near = hi != KEY_NONE && lo <= hi;
    }
    return in;
}

// Groups that are no runs of 2^n lanes: the row's values pass through shared
// memory, where 1 << lp_log2 lanes take a group; its stride gsp is that number
// modulo 32, so that no two lanes meet in a bank.
template <int V>
__device__ __forceinline__ void group_top2(const RouteParams &p, const float *s, float *s_row, int lane, float &t1,
                                           float &t2) {
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = expert_of<V>(lane, v);
        if (e < p.E) s_row[e + ((e * p.gmul) >> 20) * (p.gsp - p.gs)] = s[v];
    }
    __syncwarp();
    const int g = lane >> p.lp_log2;
    t1 = t2 = -INFINITY;
    if (g < p.G)
        for (int i = lane & ((1 << p.lp_log2) - 1); i < p.gs; i += 1 << p.lp_log2) {
            const float v = s_row[g * p.gsp + i];
            t2 = fmaxf(t2, fminf(t1, v));
            t1 = fmaxf(t1, v);
        }
    join_top2(t1, t2, p.lp_log2);
}

// The row's experts in the order of their keys, one per call of next(): a
// warp-wide maximum over the lanes' lists of their best D keys; a lane that has
// given its list away makes the next one.  A key's low bits hold the expert
// (as MASK - e: the lower expert first), so keys differ and the maximum tells
// whose it is; a value's own low bits are lost, which matters to fp32 values
// only (a bf16 or fp16 value has at least 13 zero bits).
template <int V> struct Chooser {
    static constexpr int D = V <= 4 ? V : 2;
    static constexpr uint32_t MASK = 32 * V - 1;
    const uint32_t *key;
    uint32_t k[D];
    uint32_t best = KEY_NONE;

    static __device__ __forceinline__ uint32_t key_of(float f, int lane, int v) {
        return (float_key(f) & ~MASK) | (MASK - expert_of<V>(lane, v));
    }
    static __device__ __forceinline__ int expert(uint32_t key) { return static_cast<int>(MASK - (key & MASK)); }
    static __device__ __forceinline__ bool is_open(uint32_t key) { return (key | MASK) > KEY_CLOSED; }
    __device__ __forceinline__ explicit Chooser(const uint32_t *keys) : key(keys) { list(~0u); }
    // the largest D keys below limit
    __device__ __forceinline__ void list(uint32_t limit) {
#pragma unroll
        for (int d = 0; d < D; ++d) k[d] = KEY_NONE;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t x = key[v] < limit ? key[v] : KEY_NONE;
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const uint32_t hi = max(k[d], x);
                x = min(k[d], x);
                k[d] = hi;
            }
        }
    }
    __device__ __forceinline__ void next() {
        best = __reduce_max_sync(FULL, k[0]);
        if (k[0] == best) {
#pragma unroll
            for (int d = 0; d + 1 < D; ++d) k[d] = k[d + 1];
            k[D - 1] = KEY_NONE;
        }
        if (D < V && __any_sync(FULL, k[0] == KEY_NONE)) {
            if (k[0] == KEY_NONE) list(best);  // what is left of every lane is below best
        }
    }
};

// The same for the rows that are ordered by 64-bit keys: ties are exact ones.
struct Best64 {
    uint64_t key;
    int e;
};
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(FULL, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(FULL, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
template <int V> __device__ __forceinline__ Best64 take_best64(uint64_t *key, int lane) {
    uint64_t k = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (key[v] > k) { k = key[v]; at = v; }
    Best64 b;
    b.key = warp_max_key(k);
    const int src = __ffs(__ballot_sync(FULL, k == b.key)) - 1;
    b.e = __shfl_sync(FULL, expert_of<V>(lane, at), src);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (b.e == expert_of<V>(lane, v)) key[v] = 0;
    return b;
}

// 64-bit keys, ordered like the doubles; NaN and -inf are closed.
constexpr uint64_t KEY64_CLOSED = 0x000FFFFFFFFFFFFFull;
__device__ __forceinline__ uint64_t double_key(double s) {
    if (!(s > -INFINITY)) return KEY64_CLOSED;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_double(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// One row whose experts are chosen by their 64-bit selection scores, from the
// logits to the outputs.  Comparisons are of integer keys: fp64 instructions
// are slow here (two lanes a cycle) and the row is waited for.
template <typename T, int V>
__device__ __noinline__ void route_row_f64(const RouteParams &p, int64_t t, int lane, int32_t *s_hist) {
    const T *row = static_cast<const T *>(p.logits) + t * p.ld;
    alignas(16) T raw[V];
    load_row<T, V>(row, p.E, lane, p.vec, raw);
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = to_f32(raw[v]);
        nan = nan || x != x || (x == INFINITY && p.score == KOSMOS_SCORE_SOFTMAX);
    }
    nan = __any_sync(FULL, nan);
    const bool by_logit = p.bias == nullptr;
    double m = 0.0, z = 1.0;
    if (p.score == KOSMOS_SCORE_SOFTMAX) {
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) top = fmaxf(top, to_f32(raw[v]));
        m = key_float(__reduce_max_sync(FULL, float_key(top)));
        z = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (to_f32(raw[v]) > -INFINITY) z += exp(static_cast<double>(to_f32(raw[v])) - m);
        z = warp_sum(z);
    }
    uint64_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = expert_of<V>(lane, v);
        const double x = to_f32(raw[v]);
        key[v] = KEY64_CLOSED;
        if (x > -INFINITY) {
            double s = p.score == KOSMOS_SCORE_SOFTMAX ? exp(x - m) / z : 1.0 / (1.0 + exp(-x));
            if (!by_logit) s += static_cast<double>(p.bias[e]);
            key[v] = double_key(s);
        }
    }
    if (p.GK < p.G) {
        double score = -INFINITY;  // lane g: the score of group g
        for (int g = 0; g < p.G; ++g) {
            // the group's best two keys: the best two of every lane, then of the warp
            uint64_t k1 = 0, k2 = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = expert_of<V>(lane, v) - g * (p.E / p.G);
                const uint64_t k = e >= 0 && e < p.E / p.G ? key[v] : 0;
                if (k > k1) { k2 = k1; k1 = k; }
                else if (k > k2) k2 = k;
            }
            const uint64_t b1 = warp_max_key(k1);
            const int src = __ffs(__ballot_sync(FULL, k1 == b1)) - 1;
            const uint64_t b2 = warp_max_key(lane == src ? k2 : k1);
            double t = key_double(b1);
            if (p.group_top == 2 && b2 > KEY64_CLOSED) t += key_double(b2);
            if (lane == g) score = t;
        }
        int rank = 0;
        const uint64_t mine = double_key(score);
        for (int g = 0; g < p.G; ++g) {
            const uint64_t o = __shfl_sync(FULL, mine, g);
            rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        const uint32_t open = __ballot_sync(FULL, lane < p.G && rank < p.GK);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V>(lane, v);
            if (e < p.E && !((open >> (e / (p.E / p.G))) & 1u)) key[v] = KEY64_CLOSED;
        }
    }
    if (by_logit) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > KEY64_CLOSED) key[v] = double_key(static_cast<double>(to_f32(raw[v])));
    }
    int my_e = 0;
    bool my_open = false;
    for (int j = 0; j < p.k; ++j) {
        const Best64 b = take_best64<V>(key, lane);
        if (lane == j) { my_e = b.e; my_open = b.key > KEY64_CLOSED; }
    }
    const bool mine = lane < p.k;
    float g = route_gate(p, 16, mine ? to_f32(row[my_e]) : 0.f, mine && my_open, static_cast<float>(m), static_cast<float>(z));
    if (nan) g = NAN;
    if (mine) {
        p.idx[t * p.k + lane] = my_e;
        p.gate[t * p.k + lane] = g;
        if (p.counts != nullptr) atomicAdd(&s_hist[my_e], 1);
    }
}

// A warp takes p.rows consecutive rows at a time, with p.slots lanes for each
// (a power of two, at least k): the rows are ordered one after the other, and
// the rest is done for them together, lane r * slots + j holding row r's j-th
// candidate.  Candidates beyond the k-th are taken while their keys differ from
// the k-th's in the expert alone; the candidates are then ranked by their
// scores in full.  What the scores' errors leave open goes to a list (LATER rows
// per warp) and is done at the end by route_row_f64: a call here would keep
// the loop's values out of registers.
constexpr int LATER = 16;

template <typename T, int V, int MODE>
__global__ void __launch_bounds__(ROUTE_THREADS, V <= 8 ? MINB : 1) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr bool EXACT = MODE == BY_LOGIT && sizeof(T) == 2;  // keys hold their values whole
    using Choose = Chooser<V>;
    extern __shared__ int32_t s_mem[];
    __shared__ int64_t s_later[ROUTE_WARPS][LATER];
    int32_t *s_hist = s_mem;                                           // [E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *s_row = reinterpret_cast<float *>(s_mem + p.hist_words) + warp * p.row_words;
    if (p.counts != nullptr) {
        for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) s_hist[i] = 0;
        __syncthreads();
    }
    const bool softmax = MODE == BY_SOFTMAX || (MODE == BY_LOGIT && p.score == KOSMOS_SCORE_SOFTMAX);
    const bool need_z = MODE == BY_SOFTMAX || (softmax && !p.renorm);
    const T *logits = static_cast<const T *>(p.logits);
    const int seg = lane / p.slots, slot = lane % p.slots;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROUTE_WARPS * p.rows;
    int64_t t0 = (static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp) * p.rows;
    while (t0 < p.T) {
        float bias[V];
        if (MODE != BY_LOGIT) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = expert_of<V>(lane, v);
                bias[v] = p.bias != nullptr && e < p.E ? p.bias[e] : 0.f;
            }
        }
        int later = 0;
        alignas(16) T next[V];
        load_row<T, V>(logits + t0 * p.ld, p.E, lane, p.vec, next);
        for (; t0 < p.T && later <= LATER - p.rows; t0 += stride) {
            uint32_t my_key = KEY_NONE, border = KEY_NONE;
            float my_m = 0.f, my_z = 1.f;
            bool my_nan = false, my_near = false;
            int most = p.k;  // candidates of the longest row
            const int rows = p.T - t0 < p.rows ? static_cast<int>(p.T - t0) : p.rows;
#pragma unroll 1
            for (int r = 0; r < rows; ++r) {
                float x[V];
#pragma unroll
                for (int v = 0; v < V; ++v) x[v] = to_f32(next[v]);
                const int64_t tn = r + 1 < rows ? t0 + r + 1 : t0 + stride;
                if (tn < p.T) load_row<T, V>(logits + tn * p.ld, p.E, lane, p.vec, next);
                bool nan = false;
                float m = -INFINITY, z = 1.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    nan = nan || x[v] != x[v];
                    if (MODE != BY_SIGMOID) x[v] = fmaxf(x[v], -INFINITY);  // NaN: closed
                }
                if (softmax) {
#pragma unroll
                    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
                    nan = nan || m == INFINITY;
                }
                nan = __any_sync(FULL, nan);
                // s: what orders the experts and scores the groups; closed experts -inf
                float s[V];
                if (need_z) {
                    m = key_float(__reduce_max_sync(FULL, float_key(m)));
                    if (m == -INFINITY) m = 0.f;
                    z = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        s[v] = ex2(LOG2E * (x[v] - m));
                        z += s[v];
                    }
                    z = warp_sum(z);
                }
                const float rz = MODE == BY_SOFTMAX ? rcp(z) : 1.f;
                uint32_t key[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (MODE == BY_LOGIT) {
                        s[v] = x[v];
                    } else {
                        const float q = MODE == BY_SOFTMAX ? s[v] * rz : fast_p<BY_SIGMOID>(x[v], 0.f, 1.f);
                        s[v] = x[v] > -INFINITY ? fmaxf(q + bias[v], -INFINITY) : -INFINITY;
                    }
                    key[v] = Choose::key_of(s[v], lane, v);
                }
                bool near = false;
                if (p.GK < p.G) {
                    const float err = MODE == BY_LOGIT ? 0.f : p.group_top * (MODE == BY_SOFTMAX ? 5.3e-6f * rz : 5e-7f);
                    float t1, t2;
                    if (p.lane_groups) {
                        t1 = t2 = -INFINITY;
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            t2 = fmaxf(t2, fminf(t1, s[v]));
                            t1 = fmaxf(t1, s[v]);
                        }
                        join_top2(t1, t2, p.lp_log2);
                        if (!group_open(p, t1, t2, lane, err, near)) {
#pragma unroll
                            for (int v = 0; v < V; ++v) key[v] = Choose::key_of(-INFINITY, lane, v);
                        }
                    } else {
                        group_top2<V>(p, s, s_row, lane, t1, t2);
                        const uint32_t open = __ballot_sync(FULL, group_open(p, t1, t2, lane, err, near));
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const int e = expert_of<V>(lane, v);
                            const int g = e < p.E ? (e * p.gmul) >> 20 : 0;
                            if (!((open >> (g << p.lp_log2)) & 1u)) key[v] = Choose::key_of(-INFINITY, lane, v);
                        }
                    }
                }
                Choose c(key);
                const int first = r * p.slots;
#pragma unroll 1
                for (int j = 0; j < p.k; ++j) {
                    c.next();
                    if (lane == first + j) my_key = c.best;
                }
                if (!EXACT && p.k < p.E) {
                    const uint32_t last = c.best | Choose::MASK;
                    c.next();
                    int n = p.k;
                    for (; (c.best | Choose::MASK) == last && last > KEY_CLOSED && n < p.slots && n + 1 < p.E; ++n) {
                        if (lane == first + n) my_key = c.best;
                        c.next();
                    }
                    near = near || ((c.best | Choose::MASK) == last && last > KEY_CLOSED);
                    if (n > most) most = n;
                }
                if (seg == r) {
                    border = p.k < p.E ? c.best : KEY_NONE;
                    my_nan = nan;
                    my_near = near;
                    my_m = m;
                    my_z = z;
                }
            }
            // ---- the rows together
            const bool mine = my_key != KEY_NONE;
            const T *row = logits + (t0 + (seg < rows ? seg : 0)) * p.ld;
            const bool my_open = mine && Choose::is_open(my_key);
            const int my_e = mine ? Choose::expert(my_key) : 0;
            const float my_x = EXACT ? key_float((my_key & 0x80000000u) ? my_key & ~Choose::MASK : my_key | Choose::MASK)
                                     : to_f32(row[my_e]);
            int rank = mine ? slot : p.k;
            if (!EXACT) {
                // ranked by the score in full; equal scores keep the keys' order,
                // which is that of the experts
                const float rz = MODE == BY_SOFTMAX ? rcp(my_z) : 1.f;
                const float my_b = MODE != BY_LOGIT && p.bias != nullptr ? p.bias[my_e] : 0.f;
                const float my_p = fast_p<MODE>(my_x, my_m, rz);
                const float my_s = !my_open ? -INFINITY : MODE == BY_LOGIT ? my_x : my_p + my_b;
                const float my_err = score_error<MODE>(my_s, my_p, rz);
                bool close = false;
                rank = mine ? 0 : p.k;
                for (int o = 0; o < most; ++o) {
                    const float so = __shfl_sync(FULL, my_s, seg * p.slots + o);
                    rank += (so > my_s || (so == my_s && o < slot)) ? 1 : 0;
                    // a pair within its errors: the wider one's is at least half of their sum
                    if (MODE != BY_LOGIT) close = close || (o != slot && fabsf(so - my_s) <= 2.f * my_err);
                }
                if (MODE != BY_LOGIT && __any_sync(FULL, close && mine)) {
                    // unless they are the same logit and bias: a tie in 64 bits too
                    for (int o = 0; o < most; ++o) {
                        const int src = seg * p.slots + o;
                        const float so = __shfl_sync(FULL, my_s, src), eo = __shfl_sync(FULL, my_err, src);
                        const float xo = __shfl_sync(FULL, my_x, src), bo = __shfl_sync(FULL, my_b, src);
                        const bool oo = __shfl_sync(FULL, static_cast<int>(my_open), src) != 0;
                        if (my_open && oo && !(fabsf(so - my_s) > my_err + eo) && !(xo == my_x && bo == my_b)) my_near = true;
                    }
                }
                if (mine && rank == p.k - 1 && my_open && Choose::is_open(border)) {
                    // everything that is left is at most the border's value, its p at most 1 / z
                    const float sb = key_float(border | Choose::MASK);
                    if (!(my_s - sb > my_err + score_error<MODE>(sb, rz, rz))) my_near = true;
                }
                uint32_t nb = __ballot_sync(FULL, my_near && mine);
                for (int r = 0; nb != 0u && r < rows; ++r) {
                    if (((nb >> (r * p.slots)) & ((1u << p.slots) - 1u)) == 0u) continue;
                    if (lane == 0) s_later[warp][later] = t0 + r;
                    ++later;
                    if (seg == r) rank = p.k;  // not now
                }
            }
            float g = route_gate(p, p.slots, my_x, my_open && rank < p.k, my_m, my_z);
            if (my_nan) g = NAN;
            if (rank < p.k) {
                const int64_t at = (t0 + seg) * p.k + rank;
                p.idx[at] = my_e;
                p.gate[at] = g;
                if (p.counts != nullptr) atomicAdd(&s_hist[my_e], 1);
            }
        }
        __syncwarp();
        for (int i = 0; i < later; ++i) route_row_f64<T, V>(p, s_later[warp][i], lane, s_hist);
        __syncwarp();
    }
    if (p.counts == nullptr) return;
    __syncthreads();
    if (gridDim.x == 1) {
        for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) p.counts[i] = s_hist[i];
        return;
    }
    // blocks add their counts into the workspace (integers: any order gives
    // the same sums); the last one hands them out and leaves zeros
    for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS)
        if (s_hist[i] != 0) atomicAdd(&p.acc[i], s_hist[i]);
    __threadfence();
    __syncthreads();
    __shared__ int s_last;
    if (threadIdx.x == 0) s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) {
        p.counts[i] = __ldcg(&p.acc[i]);
        p.acc[i] = 0;
    }
    if (threadIdx.x == 0) *p.ticket = 0u;
}

template <typename T, int MODE> kosmos_status launch_route_m(const RouteParams &q, int sms, cudaStream_t stream) {
    RouteParams p = q;
    const int v = p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
    const int es = static_cast<int>(sizeof(T));
    const int w = v * es < 16 ? v : 16 / es;  // values per load
    p.vec = p.E % w == 0 && reinterpret_cast<uintptr_t>(p.logits) % (w * es) == 0 && p.ld * es % (w * es) == 0;
    // several rows per warp share the gates' arithmetic, once every warp has
    // some; before that a row's latency counts
    p.slots = MODE == BY_LOGIT && es == 2 && p.k <= 8 ? 8 : 16;
    p.rows = p.T >= ROUTE_ROWS_FROM * static_cast<int64_t>(sms) ? 32 / p.slots : 1;
    int64_t blocks = cdiv(p.T, ROUTE_WARPS * p.rows);
    if (blocks > MINB * static_cast<int64_t>(sms)) blocks = MINB * static_cast<int64_t>(sms);
    const dim3 grid(static_cast<unsigned>(blocks));
    p.hist_words = p.counts != nullptr ? p.E : 0;
    p.row_words = 0;
    p.lane_groups = false;
    if (p.GK < p.G) {
        p.gs = p.E / p.G;
        p.lane_groups = p.gs % v == 0 && (p.gs / v & (p.gs / v - 1)) == 0;
        p.lp_log2 = 0;
        if (p.lane_groups) {
            while (v << p.lp_log2 < p.gs) ++p.lp_log2;
        } else {
            p.gmul = ((1 << 20) + p.gs - 1) / p.gs;  // e * gmul >> 20 = e / gs for e < 1024
            while ((p.G << (p.lp_log2 + 1)) <= 32) ++p.lp_log2;
            p.gsp = p.gs + ((1 << p.lp_log2) - p.gs % 32 + 32) % 32;
            p.row_words = p.G * p.gsp;
        }
    }
    const size_t smem = 4ull * (p.hist_words + ROUTE_WARPS * p.row_words);
    switch (v) {
        case 2: route_kernel<T, 2, MODE><<<grid, ROUTE_THREADS, smem, stream>>>(p); break;
        case 4: route_kernel<T, 4, MODE><<<grid, ROUTE_THREADS, smem, stream>>>(p); break;
        case 8: route_kernel<T, 8, MODE><<<grid, ROUTE_THREADS, smem, stream>>>(p); break;
        case 16: route_kernel<T, 16, MODE><<<grid, ROUTE_THREADS, smem, stream>>>(p); break;
        default: route_kernel<T, 32, MODE><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? KOSMOS_OK : KOSMOS_ERR_CUDA;
}

template <typename T> kosmos_status launch_route_t(const RouteParams &p, int sms, cudaStream_t stream) {
    if (p.bias == nullptr && !(p.GK < p.G && p.group_top == 2)) return launch_route_m<T, BY_LOGIT>(p, sms, stream);
    if (p.score == KOSMOS_SCORE_SIGMOID) return launch_route_m<T, BY_SIGMOID>(p, sms, stream);
    return launch_route_m<T, BY_SOFTMAX>(p, sms, stream);
}

struct RouteBwdParams {
    const void *logits;
    const int32_t *idx;
    const float *gate, *dgate;
    void *dlogits;
    int64_t T, ld, ldd;
    int E, k, score, renorm;
    float scale;
};

// One warp per token.
template <typename T>
__global__ void __launch_bounds__(ROUTE_THREADS) route_bwd_kernel(const __grid_constant__ RouteBwdParams p) {
    extern __shared__ float s_rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *srow = s_rows + warp * p.E;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * ROUTE_WARPS) {
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        T *out = static_cast<T *>(p.dlogits) + t * p.ldd;
        const int e = lane < p.k ? p.idx[t * p.k + lane] : -1;
        const bool ok = e >= 0 && e < p.E;
        const float g = ok ? p.gate[t * p.k + lane] : 0.f;
        const float dg = ok ? p.dgate[t * p.k + lane] : 0.f;
        float gdg = g * dg;
        if (g == 0.f) gdg = 0.f;  // a closed pick: no gradient, whatever dg holds
        const float D = warp_sum(gdg);
        float d = gdg;
        if (p.renorm && g != 0.f) d = g * (dg - D / p.scale);
        if (p.score == KOSMOS_SCORE_SIGMOID && ok && g != 0.f) d *= 1.0f / (1.0f + expf(to_f32(row[e])));
        const bool full = p.score == KOSMOS_SCORE_SOFTMAX && !p.renorm;
        for (int i = lane; i < p.E; i += 32) srow[i] = 0.f;
        __syncwarp();
        if (ok) srow[e] = d;
        __syncwarp();
        float m = -INFINITY, z = 0.f;
        if (full) {
            for (int i = lane; i < p.E; i += 32) m = fmaxf(m, to_f32(row[i]));
            m = warp_max(m);
            for (int i = lane; i < p.E; i += 32) z += expf(to_f32(row[i]) - m);
            z = warp_sum(z);
        }
        for (int i = lane; i < p.E; i += 32) {
            float v = srow[i];
            if (full && D != 0.f) v -= D * (expf(to_f32(row[i]) - m) / z);  // D = 0 also where every pick is closed
            out[i] = from_f32<T>(v);
        }
        __syncwarp();
    }
}

template <typename T> kosmos_status launch_route_bwd_t(const RouteBwdParams &p, int sms, cudaStream_t stream) {
    int64_t blocks = cdiv(p.T, ROUTE_WARPS);
    if (blocks > 4ll * sms) blocks = 4ll * sms;
    route_bwd_kernel<T><<<static_cast<unsigned>(blocks), ROUTE_THREADS, sizeof(float) * ROUTE_WARPS * p.E, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KOSMOS_OK : KOSMOS_ERR_CUDA;
}

}  // namespace

size_t route_workspace_bytes(int E) { return 256 + static_cast<size_t>(align_up(4ll * E, 256)); }

kosmos_status launch_route(const RouteLaunch &L, cudaStream_t stream) {
    if (L.T == 0) {
        if (L.counts == nullptr) return KOSMOS_OK;
        return cudaMemsetAsync(L.counts, 0, 4ull * L.E, stream) == cudaSuccess ? KOSMOS_OK : KOSMOS_ERR_CUDA;
    }
    RouteParams p = {};
    p.logits = L.logits; p.bias = L.bias; p.idx = L.idx; p.gate = L.gate; p.counts = L.counts;
    p.ticket = L.counts ? &static_cast<WsHeader *>(L.ws)->done_ctas : nullptr;
    p.acc = L.counts ? reinterpret_cast<int32_t *>(static_cast<uint8_t *>(L.ws) + 256) : nullptr;
    p.T = L.T; p.ld = L.ld; p.E = L.E; p.k = L.r.topk; p.G = L.r.n_groups; p.GK = L.r.topk_groups;
    p.group_top = L.r.group_top; p.score = L.r.score; p.renorm = L.r.renorm; p.scale = L.r.scale;
    if (L.dtype == KOSMOS_BF16) return launch_route_t<__nv_bfloat16>(p, L.sms, stream);
    if (L.dtype == KOSMOS_FP16) return launch_route_t<__half>(p, L.sms, stream);
    return launch_route_t<float>(p, L.sms, stream);
}

kosmos_status launch_route_bwd(const RouteBwdLaunch &L, cudaStream_t stream) {
    RouteBwdParams p;
    p.logits = L.logits; p.idx = L.idx; p.gate = L.gate; p.dgate = L.dgate; p.dlogits = L.dlogits;
    p.T = L.T; p.ld = L.ld; p.ldd = L.ldd; p.E = L.E; p.k = L.r.topk; p.score = L.r.score; p.renorm = L.r.renorm;
    p.scale = L.r.scale;
    if (L.dtype == KOSMOS_BF16) return launch_route_bwd_t<__nv_bfloat16>(p, L.sms, stream);
    if (L.dtype == KOSMOS_FP16) return launch_route_bwd_t<__half>(p, L.sms, stream);
    return launch_route_bwd_t<float>(p, L.sms, stream);
}

}  // namespace kosmos
