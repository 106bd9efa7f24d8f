// route_bf16.cu -- the router's forward kernels for bf16 logits.
#include "route_fwd.cuh"

namespace kosmos {

kosmos_status launch_route_bf16(const RouteParams &p, int sms, cudaStream_t stream) {
    return launch_route_t<__nv_bfloat16>(p, sms, stream);
}

}  // namespace kosmos
