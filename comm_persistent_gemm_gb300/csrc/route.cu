// route.cu -- the router of an expert layer on its own: the forward's dispatch by
// type (its kernel is in route_fwd.cuh) and the gradient of the gates with
// respect to the logits.
#include "route.cuh"

namespace kosmos {

namespace {

constexpr int BWD_WARPS = 8;
constexpr int BWD_THREADS = BWD_WARPS * 32;

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
__global__ void __launch_bounds__(BWD_THREADS) route_bwd_kernel(const __grid_constant__ RouteBwdParams p) {
    extern __shared__ float s_rows[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *srow = s_rows + warp * p.E;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * BWD_WARPS + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * BWD_WARPS) {
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        T *out = static_cast<T *>(p.dlogits) + t * p.ldd;
        const int e = lane < p.k ? p.idx[t * p.k + lane] : -1;
        const bool ok = e >= 0 && e < p.E;
        const float g = ok ? p.gate[t * p.k + lane] : 0.f;
        const float dg = ok ? p.dgate[t * p.k + lane] : 0.f;
        float gdg = g * dg;
        if (g == 0.f) gdg = 0.f;  // a closed pick: no gradient, whatever dg holds
        const float D = row_sum<32>(gdg);
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
            m = row_max<32>(m);
            for (int i = lane; i < p.E; i += 32) z += expf(to_f32(row[i]) - m);
            z = row_sum<32>(z);
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
    int64_t blocks = cdiv(p.T, BWD_WARPS);
    if (blocks > 4ll * sms) blocks = 4ll * sms;
    route_bwd_kernel<T><<<static_cast<unsigned>(blocks), BWD_THREADS, sizeof(float) * BWD_WARPS * p.E, stream>>>(p);
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
    if (L.dtype == KOSMOS_BF16) return launch_route_bf16(p, L.sms, stream);
    if (L.dtype == KOSMOS_FP16) return launch_route_fp16(p, L.sms, stream);
    return launch_route_fp32(p, L.sms, stream);
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
