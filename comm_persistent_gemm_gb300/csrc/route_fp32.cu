// route_fp32.cu -- the router's forward kernels for fp32 logits.
#include "route_fwd.cuh"

namespace kosmos {

kosmos_status launch_route_fp32(const RouteParams &p, int sms, cudaStream_t stream) {
    return launch_route_t<float>(p, sms, stream);
}

}  // namespace kosmos
