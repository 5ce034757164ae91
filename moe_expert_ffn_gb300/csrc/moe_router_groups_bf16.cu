// moe_router_groups_bf16.cu -- routing limited to groups of experts, bf16 logits.
#include "moe_router_groups.cuh"

namespace moe {

cudaError_t launch_router_groups_bf16(const RouterParams &p, bool loss, int ctas, cudaStream_t s) {
    return RunGrouped<bf16>{p, loss, ctas, s}.run();
}

}  // namespace moe
