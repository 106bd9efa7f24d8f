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

template <typename T, int V>
__global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int WMAX = 16 / static_cast<int>(sizeof(T));
    constexpr int W = V < WMAX ? V : WMAX;
    extern __shared__ int32_t s_hist[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.counts != nullptr) {
        for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) s_hist[i] = 0;
        __syncthreads();
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * ROUTE_WARPS) {
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        int my_e = 0;
        bool my_open = false;
        choose_f64<T, V, W>(p, row, lane, my_e, my_open);
        bool nan = false;
        float m = -INFINITY, z = 0.f;
        for (int e = lane; e < p.E; e += 32) {
            const float x = to_f32(row[e]);
            nan = nan || isnan(x) || (x == INFINITY && p.score == KOSMOS_SCORE_SOFTMAX);
            m = fmaxf(m, x);
        }
        nan = __any_sync(FULL, nan);
        if (p.score == KOSMOS_SCORE_SOFTMAX && !p.renorm) {
            m = warp_max(m);
            for (int e = lane; e < p.E; e += 32) z += expf(to_f32(row[e]) - m);
            z = warp_sum(z);
        }
        const bool mine = lane < p.k;
        const float x = mine ? to_f32(row[my_e]) : 0.f;
        float g = route_gate(p, x, mine && my_open, m, z);
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

template <typename T> kosmos_status launch_route_t(const RouteParams &p, int sms, cudaStream_t stream) {
    int64_t blocks = cdiv(p.T, ROUTE_WARPS);
    if (blocks > 4ll * sms) blocks = 4ll * sms;
    const dim3 grid(static_cast<unsigned>(blocks));
    const size_t smem = p.counts != nullptr ? 4ull * p.E : 0;
    if (p.E <= 64) route_kernel<T, 2><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    else if (p.E <= 128) route_kernel<T, 4><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    else if (p.E <= 256) route_kernel<T, 8><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    else if (p.E <= 512) route_kernel<T, 16><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    else route_kernel<T, 32><<<grid, ROUTE_THREADS, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KOSMOS_OK : KOSMOS_ERR_CUDA;
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
    RouteParams p;
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
