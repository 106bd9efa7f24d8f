// route_fp16.cu -- the router's forward kernels for fp16 logits.
#include "route_fwd.cuh"

namespace kosmos {

kosmos_status launch_route_fp16(const RouteParams &p, int sms, cudaStream_t stream) {
    return launch_route_t<__half>(p, sms, stream);
}

}  // namespace kosmos
