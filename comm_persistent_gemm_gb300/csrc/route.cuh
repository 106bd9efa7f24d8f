// route.cuh -- what the router's forward and backward kernels share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace kosmos {

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
    bool vec;                         // pieces of a row are loaded whole
    int hist_words, row_words;        // shared memory: counts, then a row of values (groups only)
    int gs, gsp, gmul;                // group size, its stride in shared memory, division by gs
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Maximum and sum over the L lanes of a row.
template <int L> __device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, d));
    return v;
}
template <int L> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(FULL, v, d));
    return v;
}
template <int L, typename F> __device__ __forceinline__ F row_sum(F v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
    return v;
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

// Which of a row's values a lane holds: pieces of W consecutive experts (one
// load of up to 16 bytes), the row's lanes side by side.
template <typename T, int L, int V> struct Layout {
    static constexpr int W = V * sizeof(T) < 16 ? V : 16 / static_cast<int>(sizeof(T));
    static __device__ __forceinline__ int expert(int l, int v) { return (v / W) * L * W + l * W + v % W; }
    // the values as floats; beyond E: -inf
    static __device__ __forceinline__ void load(const T *row, int E, int l, bool vec, float *x) {
#pragma unroll
        for (int c = 0; c < V; c += W) {
            const int e0 = expert(l, c);
            alignas(16) T r[W];
            if (vec) {
                if (e0 < E) {
                    if constexpr (W * sizeof(T) == 16)
                        *reinterpret_cast<uint4 *>(r) = *reinterpret_cast<const uint4 *>(row + e0);
                    else
                        *reinterpret_cast<uint2 *>(r) = *reinterpret_cast<const uint2 *>(row + e0);
                    static_assert(W * sizeof(T) >= 8, "a piece is 8 or 16 bytes");
                }
#pragma unroll
                for (int i = 0; i < W; ++i) x[c + i] = e0 < E ? to_f32(r[i]) : -INFINITY;
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) x[c + i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
            }
        }
    }
};

// The forward launch for one type of logits (route_bf16.cu, route_fp16.cu, route_fp32.cu).
kosmos_status launch_route_bf16(const RouteParams &p, int sms, cudaStream_t stream);
kosmos_status launch_route_fp16(const RouteParams &p, int sms, cudaStream_t stream);
kosmos_status launch_route_fp32(const RouteParams &p, int sms, cudaStream_t stream);

}  // namespace kosmos
