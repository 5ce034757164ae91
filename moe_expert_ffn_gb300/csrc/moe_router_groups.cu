// moe_router_groups.cu -- routing limited to groups of experts, f32 logits.
#include "moe_router_groups.cuh"

namespace moe {

cudaError_t launch_router_groups_f32(const RouterParams &p, bool loss, int ctas, cudaStream_t s) {
    return RunGrouped<float>{p, loss, ctas, s}.run();
}

}  // namespace moe
