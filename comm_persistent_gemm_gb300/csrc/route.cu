// route.cu -- the router of an expert layer on its own: topk experts and their
// gates from a [tokens, experts] score matrix (softmax or sigmoid scores, a
// bias that takes part in the choice only, groups of experts of which the best
// stay open, renormalised and scaled gates, tokens per expert), and the
// gradient of the gates with respect to the logits.
//
// One warp per token; lane l holds V of the row's values.  The choice is k
// rounds of a warp-wide maximum; what decides it is an order that ties break
// towards the lower expert, so the result is a function of the row alone.
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
    int gs, gsp, gmul, lp_log2;       // group size, its stride in shared memory, division by gs, lanes per group
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The expert of lane l's value v: runs of W consecutive experts per lane.
template <int V, int W> __device__ __forceinline__ int expert_of(int lane, int v) {
    return (v / W) * 32 * W + lane * W + v % W;
}

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmax(v, __shfl_xor_sync(FULL, v, d));
    return v;
}
template <typename F> __device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
    return v;
}

// (value, index) pairs ordered by descending value, then ascending index.
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) { return a > b || (a == b && ia < ib); }

// Chooses the row's experts by their 64-bit selection scores; lane j < k gets
// the j-th expert and whether it is open.
template <typename T, int V, int W>
__device__ __noinline__ void choose_f64(const RouteParams &p, const T *row, int lane, int &my_e, bool &my_open) {
    double s[V];
    double m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = expert_of<V, W>(lane, v);
        const float x = e < p.E ? to_f32(row[e]) : -INFINITY;
        s[v] = x;
        m = fmax(m, s[v]);  // fmax skips NaN
    }
    // without a bias s rises with the logit, which then orders the experts
    // exactly; a sum of two scores needs the scores themselves
    const bool by_logit = p.bias == nullptr;
    const bool scores = !by_logit || (p.GK < p.G && p.group_top == 2);
    if (!scores) {
    } else if (p.score == KOSMOS_SCORE_SOFTMAX) {
        m = warp_max(m);
        double z = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (!isnan(s[v])) z += exp(s[v] - m);
        z = warp_sum(z);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = s[v] == -INFINITY ? -INFINITY : exp(s[v] - m) / z;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = s[v] == -INFINITY ? -INFINITY : 1.0 / (1.0 + exp(-s[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = expert_of<V, W>(lane, v);
        if (p.bias != nullptr && e < p.E) s[v] += static_cast<double>(p.bias[e]);
        if (isnan(s[v])) s[v] = -INFINITY;
    }
    if (p.GK < p.G) {
        const int gs = p.E / p.G;
        double score = -INFINITY;  // lane g: the score of group g
        for (int g = 0; g < p.G; ++g) {
            double t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = expert_of<V, W>(lane, v);
                if (e >= g * gs && e < (g + 1) * gs) {
                    if (s[v] > t1) { t2 = t1; t1 = s[v]; }
                    else if (s[v] > t2) t2 = s[v];
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const double o1 = __shfl_xor_sync(FULL, t1, d), o2 = __shfl_xor_sync(FULL, t2, d);
                t2 = fmax(fmin(t1, o1), fmax(t2, o2));
                t1 = fmax(t1, o1);
            }
            if (p.group_top == 2 && t2 != -INFINITY) t1 += t2;
            if (lane == g) score = t1;
        }
        int rank = 0;
        for (int g = 0; g < p.G; ++g) {
            const double o = __shfl_sync(FULL, score, g);
            if (before(o, g, score, lane)) ++rank;
        }
        const uint32_t open = __ballot_sync(FULL, lane < p.G && rank < p.GK);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V, W>(lane, v);
            if (e < p.E && !((open >> (e / gs)) & 1u)) s[v] = -INFINITY;
            else if (e < p.E && by_logit && s[v] != -INFINITY) s[v] = to_f32(row[e]);
        }
    }
    double last = INFINITY;
    int last_e = -1;
    for (int j = 0; j < p.k; ++j) {
        double b = -INFINITY;
        int be = 0x7FFFFFFF;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V, W>(lane, v);
            if (e < p.E && before(last, last_e, s[v], e) && before(s[v], e, b, be)) { b = s[v]; be = e; }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const double o = __shfl_xor_sync(FULL, b, d);
            const int oe = __shfl_xor_sync(FULL, be, d);
            if (before(o, oe, b, be)) { b = o; be = oe; }
        }
        if (lane == j) { my_e = be; my_open = b != -INFINITY; }
        last = b;
        last_e = be;
    }
}

// The gates of the chosen experts (lane j < k: expert of logit x, open or
// closed).  m, z: the row's maximum and sum of exponentials (softmax without
// renorm).  Ratios of p are taken relative to the largest chosen one, so that
// small scores keep their precision.
__device__ __forceinline__ float route_gate(const RouteParams &p, float x, bool open, float m, float z) {
    if (!p.renorm) {
        if (!open) return 0.f;
        return p.scale * (p.score == KOSMOS_SCORE_SOFTMAX ? expf(x - m) / z : 1.0f / (1.0f + expf(-x)));
    }
    float top = open ? x : -INFINITY;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
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
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
    return open ? p.scale * (w / sum) : 0.f;
}

// ------------------------------------------------------------ fp32 choice
// How a kernel orders a row's experts:
//   BY_LOGIT16  without a bias, 16-bit logits: the key holds the logit (19 bits
//               order a bf16 or fp16 value) and the expert, so keys differ and
//               one warp-wide maximum finds value and expert together;
//   BY_LOGIT32  without a bias, fp32 logits: the key is the logit;
//   BY_SCORE    the fp32 selection score.  Rows in which two neighbours in the
//               order, or the groups either side of the border, are closer
//               than the scores' rounding error are chosen again in 64 bits.
enum RouteMode : int { BY_LOGIT16 = 0, BY_LOGIT32 = 1, BY_SCORE = 2 };

// Order-preserving map of floats to unsigned integers (-0 as +0); every real
// expert's key is above KEY_NONE, closed ones have the key of -inf.
constexpr uint32_t KEY_NONE = 0u, KEY_CLOSED = 0x007FFFFFu, LOW13 = 0x1FFFu;
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Row t's values: runs of W consecutive experts per lane, in one load each
// where rows start on multiples of the run.  Beyond E: -inf.
template <typename T, int V, int W>
__device__ __forceinline__ void load_row(const T *row, int E, int lane, bool vec, float *x) {
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const int e0 = c * 32 * W + lane * W;
        alignas(16) T r[W];
        if (vec) {
            if (e0 < E) {
                if constexpr (sizeof(r) == 16) *reinterpret_cast<uint4 *>(r) = *reinterpret_cast<const uint4 *>(row + e0);
                else if constexpr (sizeof(r) == 8) *reinterpret_cast<uint2 *>(r) = *reinterpret_cast<const uint2 *>(row + e0);
                else *reinterpret_cast<uint32_t *>(r) = *reinterpret_cast<const uint32_t *>(row + e0);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) x[c * W + i] = e0 < E ? to_f32(r[i]) : -INFINITY;
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) x[c * W + i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
        }
    }
}

// Bounds on the distance between an fp32 score and the 64-bit one.  Sigmoid:
// the fast exponential is off by 2 + 1.2 |x| steps, which p (1 - p) brings
// under 6e-8; sum and division 3e-7 p; the bias' addition 6e-8 |s|.  Softmax:
// e^-y of a term y below the maximum is off by (2.5 + 1.7 y) steps, at most 3e-7
// of the largest term; the row's sum by 5e-6 (its terms' errors weigh
// at most ln 1024, and 37 additions); the bias as above.
__device__ __forceinline__ float score_error(int score, float s, float p, float z) {
    return (score == KOSMOS_SCORE_SIGMOID ? 5e-7f : 3e-7f / z + 5e-6f * p) + 1.2e-7f * fabsf(s);
}

// The groups that stay open, as a bit mask, from the row's values s (closed
// experts -inf).  The values pass through shared memory, where 32 / G lanes
// (G rounded up to a power of two) take a group; its stride gsp is the lanes'
// number modulo 32, so that no two lanes meet in a bank.  err > 0: the error of
// the values of one group's score; near then tells that the border lies
// between group scores that their errors do not separate.
template <int V, int W>
__device__ __forceinline__ uint32_t open_groups(const RouteParams &p, const float *s, float *s_row, int lane,
                                                float err, bool &near) {
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = expert_of<V, W>(lane, v);
        if (e < p.E) s_row[e + ((e * p.gmul) >> 20) * (p.gsp - p.gs)] = s[v];
    }
    __syncwarp();
    const int g = lane >> p.lp_log2, sub = lane & ((1 << p.lp_log2) - 1);
    float t1 = -INFINITY, t2 = -INFINITY;
    if (g < p.G)
        for (int i = sub; i < p.gs; i += 1 << p.lp_log2) {
            const float v = s_row[g * p.gsp + i];
            t2 = fmaxf(t2, fminf(t1, v));
            t1 = fmaxf(t1, v);
        }
    for (int d = 1; d < (1 << p.lp_log2); d <<= 1) {
        const float o1 = __shfl_xor_sync(FULL, t1, d), o2 = __shfl_xor_sync(FULL, t2, d);
        t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
        t1 = fmaxf(t1, o1);
    }
    float ge = err + 2.4e-7f * fabsf(t1);  // on the group's score: two scores' errors and their sum's
    if (p.group_top == 2 && t2 != -INFINITY) {
        ge += 2.4e-7f * fabsf(t2);
        t1 += t2;
    }
    int rank = 0;
    for (int o = 0; o < p.G; ++o) {
        const float v = __shfl_sync(FULL, t1, o << p.lp_log2);
        rank += (v > t1 || (v == t1 && o < g)) ? 1 : 0;
    }
    const bool in = g < p.G && rank < p.GK, out = g < p.G && rank >= p.GK;
    if (err > 0.f) {
        float lo = in ? t1 - ge : INFINITY, hi = out && t1 != -INFINITY ? t1 + ge : -INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(FULL, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(FULL, hi, d));
        }
        near = hi != -INFINITY && !(lo > hi);
    }
    // one bit per group: every group's first lane votes
    const uint32_t b = __ballot_sync(FULL, in && sub == 0);
    uint32_t mask = b;
    if (p.lp_log2 != 0) {
        mask = 0u;
        for (int o = 0; o < p.G; ++o) mask |= ((b >> (o << p.lp_log2)) & 1u) << o;
    }
    return mask;
}

template <typename T, int V, int MODE>
__global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int WMAX = 16 / static_cast<int>(sizeof(T));
    constexpr int W = V < WMAX ? V : WMAX;
    extern __shared__ int32_t s_mem[];
    int32_t *s_hist = s_mem;                                           // [E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *s_row = reinterpret_cast<float *>(s_mem + p.hist_words) + warp * p.row_words;
    if (p.counts != nullptr) {
        for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) s_hist[i] = 0;
        __syncthreads();
    }
    const bool by_logit = MODE != BY_SCORE || p.bias == nullptr;
    const bool softmax = p.score == KOSMOS_SCORE_SOFTMAX;
    const bool need_z = softmax && (MODE == BY_SCORE || !p.renorm);
    const int rounds = p.k + ((MODE == BY_SCORE && !by_logit && p.k < p.E) ? 1 : 0);  // one more: the border's other side
    float bias[V];
    if (MODE == BY_SCORE) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V, W>(lane, v);
            bias[v] = p.bias != nullptr && e < p.E ? p.bias[e] : 0.f;
        }
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * ROUTE_WARPS) {
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        float x[V];
        load_row<T, V, W>(row, p.E, lane, p.vec, x);
        bool nan = false;
        float m = -INFINITY, z = 1.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nan = nan || x[v] != x[v] || (softmax && x[v] == INFINITY);
            m = fmaxf(m, x[v]);  // skips NaN
        }
        nan = __any_sync(FULL, nan);
        if (need_z) {
            m = warp_max(m);
            z = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) z += x[v] > -INFINITY ? __expf(x[v] - m) : 0.f;
            z = warp_sum(z);
        }
        // the row's order: s, closed experts -inf
        float s[V];
        bool near = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = x[v];
            if (MODE == BY_SCORE && !(by_logit && p.GK == p.G)) {
                s[v] = softmax ? __fdividef(__expf(x[v] - m), z) : __fdividef(1.0f, 1.0f + __expf(-x[v]));
                s[v] = x[v] > -INFINITY ? s[v] + bias[v] : -INFINITY;
            }
            s[v] = s[v] > -INFINITY ? s[v] : -INFINITY;  // NaN
        }
        uint32_t open = FULL;
        if (p.GK < p.G) {
            const float err = MODE == BY_SCORE ? p.group_top * (softmax ? 5.3e-6f / z : 5e-7f) : 0.f;
            open = open_groups<V, W>(p, s, s_row, lane, err, near);
        }
        uint32_t key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V, W>(lane, v);
            float o = MODE == BY_SCORE && by_logit && s[v] > -INFINITY ? x[v] : s[v];
            if (p.GK < p.G && !((open >> ((e * p.gmul) >> 20)) & 1u)) o = -INFINITY;
            key[v] = float_key(o);
            if (MODE == BY_LOGIT16) key[v] = (key[v] & ~LOW13) | (LOW13 - e);
            if (e >= p.E) key[v] = KEY_NONE;
        }
        // k rounds of a warp-wide maximum over every lane's best two; a lane
        // that has given both away looks for its next two
        uint32_t my_key = KEY_NONE;
        int my_e = 0;
        uint32_t k1 = KEY_NONE, k2 = KEY_NONE;
        int e1 = 0x7FFFFFFF, e2 = 0x7FFFFFFF, have = 2;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = expert_of<V, W>(lane, v);
            if (key[v] > k1) { k2 = k1; e2 = e1; k1 = key[v]; e1 = e; }
            else if (key[v] > k2) { k2 = key[v]; e2 = e; }
        }
        for (int j = 0; j < rounds; ++j) {
            const uint32_t best = __reduce_max_sync(FULL, k1);
            int e = e1;
            if (MODE != BY_LOGIT16) e = __reduce_min_sync(FULL, k1 == best ? static_cast<uint32_t>(e1) : 0x7FFFFFFFu);
            const bool won = k1 == best && (MODE == BY_LOGIT16 || e == e1);
            if (lane == j) { my_key = best; my_e = e; }
            if (won) { k1 = k2; e1 = e2; --have; }
            if (__any_sync(FULL, have == 0) && j + 1 < rounds) {
                if (have == 0) {
                    k1 = k2 = KEY_NONE;
                    e1 = e2 = 0x7FFFFFFF;
                    have = 2;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int ev = expert_of<V, W>(lane, v);
                        const bool left = key[v] < best || (MODE != BY_LOGIT16 && key[v] == best && ev > e);
                        if (left && key[v] > k1) { k2 = k1; e2 = e1; k1 = key[v]; e1 = ev; }
                        else if (left && key[v] > k2) { k2 = key[v]; e2 = ev; }
                    }
                }
            }
        }
        const bool mine = lane < p.k;
        bool my_open;
        float my_x = 0.f;
        if (MODE == BY_LOGIT16) {
            my_e = LOW13 - (my_key & LOW13);
            my_open = (my_key | LOW13) > KEY_CLOSED;
            my_x = key_float((my_key & 0x80000000u) ? my_key & ~LOW13 : my_key | LOW13);
        } else {
            my_open = my_key > KEY_CLOSED;
            if (MODE == BY_LOGIT32) my_x = key_float(my_key);
        }
        if (MODE == BY_SCORE) {
            if (lane < rounds) my_x = to_f32(row[my_e]);
            if (!by_logit) {
                // neighbours closer than their errors, unless they are the same logit
                // and bias (a tie in 64 bits too, which the index has broken)
                const float my_s = key_float(my_key), my_b = lane < rounds ? p.bias[my_e] : 0.f;
                const float my_err = score_error(p.score, my_s, fabsf(my_s - my_b), z);
                const float s2 = __shfl_down_sync(FULL, my_s, 1), err2 = __shfl_down_sync(FULL, my_err, 1);
                const float x2 = __shfl_down_sync(FULL, my_x, 1), b2 = __shfl_down_sync(FULL, my_b, 1);
                const bool open2 = __shfl_down_sync(FULL, static_cast<int>(my_open), 1) != 0;
                near = near || (lane + 1 < rounds && my_open && open2 && !(my_s - s2 > my_err + err2) &&
                                !(my_x == x2 && my_b == b2));
            }
            if (__any_sync(FULL, near)) {
                choose_f64<T, V, W>(p, row, lane, my_e, my_open);
                if (mine) my_x = to_f32(row[my_e]);
            }
        }
        float g = route_gate(p, my_x, mine && my_open, m, z);
        if (nan) g = NAN;
        if (mine) {
            p.idx[t * p.k + lane] = my_e;
            p.gate[t * p.k + lane] = g;
            if (p.counts != nullptr) atomicAdd(&s_hist[my_e], 1);
        }
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
    int64_t blocks = cdiv(p.T, ROUTE_WARPS);
    if (blocks > 4ll * sms) blocks = 4ll * sms;
    const dim3 grid(static_cast<unsigned>(blocks));
    const int v = p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
    const int w = v < 16 / static_cast<int>(sizeof(T)) ? v : 16 / static_cast<int>(sizeof(T));
    const int64_t run = w * static_cast<int64_t>(sizeof(T));
    p.vec = p.E % w == 0 && reinterpret_cast<uintptr_t>(p.logits) % run == 0 && p.ld * sizeof(T) % run == 0;
    p.hist_words = p.counts != nullptr ? p.E : 0;
    p.row_words = 0;
    if (p.GK < p.G) {
        p.gs = p.E / p.G;
        p.gmul = ((1 << 20) + p.gs - 1) / p.gs;  // e * gmul >> 20 = e / gs for e < 1024
        p.lp_log2 = 0;
        while ((p.G << (p.lp_log2 + 1)) <= 32) ++p.lp_log2;
        p.gsp = p.gs + ((1 << p.lp_log2) - p.gs % 32 + 32) % 32;
        p.row_words = p.G * p.gsp;
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
    if (p.bias != nullptr || (p.GK < p.G && p.group_top == 2)) return launch_route_m<T, BY_SCORE>(p, sms, stream);
    return launch_route_m<T, sizeof(T) == 2 ? BY_LOGIT16 : BY_LOGIT32>(p, sms, stream);
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
