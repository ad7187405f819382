// host_stubs_layer.cpp -- the launchers behind moe_layer.h replaced by stubs,
// as host_stubs.cpp does for moe_prefill.h.  Every stub reports an error: no
// CPU test reaches a launch.
#include "../../quantized_moe_expert_scatter_amd/csrc/layer_ops.h"

namespace moe {

hipError_t launch_route(const RouteArgs &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_route_balance(const RouteArgs &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_route_backward(const RouteArgs &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_combine_backward(const float *, const float *, const float *, int, int, int, float *, float *,
                                   hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_adapters(const AdapterArgs &, hipStream_t) { return hipErrorNotSupported; }

}  // namespace moe
