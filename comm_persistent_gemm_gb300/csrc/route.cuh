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

// Copies of the counts that the blocks add into: with one, 760 blocks meet at
// its addresses (1024 x 128 in 5.0 us against 4.1, 32768 x 256 in 25.2 against 24.5).
constexpr int ROUTE_SUMS = 8;

struct RouteParams {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *gate;
    int32_t *counts;
    uint32_t *ticket;   // workspace: blocks that have added their counts
    int32_t *acc;       // workspace: [ROUTE_SUMS, E] counts so far, zero between calls
    int64_t T, ld;
    int E, k, G, GK, group_top, score, renorm;
    float scale;
    // set by the launcher
    bool vec;                         // rows are loaded in 16-byte pieces
    int width, warp_words;            // shared memory: a row's values, a warp's rows
    uint32_t mask;                    // the bits of a key that hold the expert
    int gs, gmul;                     // group size, division by it
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
    if constexpr (L == 32) {
        return __reduce_max_sync(FULL, v);
    } else {
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(FULL, v, d));
        return v;
    }
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
    // The values as floats, beyond E -inf.
    static __device__ __forceinline__ void load(const T *row, int E, int l, bool vec, float *x) {
        static_assert(W * sizeof(T) >= 8, "a piece is 8 or 16 bytes");
        constexpr int NW = W * sizeof(T) / 4;  // words of a piece
        if (vec) {
            uint32_t r[V / W][NW];
#pragma unroll
            for (int c = 0; c < V / W; ++c) load_piece(r[c], row + expert(l, c * W), expert(l, c * W) < E);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float f = to_f32(reinterpret_cast<const T *>(r[v / W])[v % W]);
                x[v] = expert(l, v - v % W) < E ? f : -INFINITY;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = expert(l, v) < E ? to_f32(row[expert(l, v)]) : -INFINITY;
        }
    }
    // In order and unconditionally issued, so that a row's pieces are all on
    // their way before the first is used; zeros where not `in`.
    static __device__ __forceinline__ void load_piece(uint32_t *r, const T *p, bool in) {
        if constexpr (W * sizeof(T) == 16) {
            r[0] = r[1] = r[2] = r[3] = 0u;
            asm volatile("{ .reg .pred q; setp.ne.s32 q, %5, 0; @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4]; }"
                         : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])
                         : "l"(p), "r"(static_cast<int>(in))
                         : "memory");
        } else {
            r[0] = r[1] = 0u;
            asm volatile("{ .reg .pred q; setp.ne.s32 q, %3, 0; @q ld.global.v2.u32 {%0, %1}, [%2]; }"
                         : "+r"(r[0]), "+r"(r[1])
                         : "l"(p), "r"(static_cast<int>(in))
                         : "memory");
        }
    }
};

// The forward launch for one type of logits (route_bf16.cu, route_fp16.cu, route_fp32.cu).
kosmos_status launch_route_bf16(const RouteParams &p, int sms, cudaStream_t stream);
kosmos_status launch_route_fp16(const RouteParams &p, int sms, cudaStream_t stream);
kosmos_status launch_route_fp32(const RouteParams &p, int sms, cudaStream_t stream);

}  // namespace kosmos
