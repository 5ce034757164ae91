// moe_router_groups.cuh -- routing limited to groups of experts (definitions in include/moe.h), by the router's kernel
// (moe_router.cuh): a group has registers of its own, so its score is a reduction or two over the lanes.  Groups are then ranked
// by comparing each with the others (four lanes to a group of eight), the keys of those left out are closed, and the choice is the
// router's.  Bound by instructions as that is: 32767 tokens of 256 f32 logits, 4 of 8 groups, 8 chosen: by the largest logit 26.0
// us (without groups 18.7), by scores with a bias and a group's two best 38.8 (21.0), 802 warp instructions a token; reading the
// logits alone takes 5.3.  128 tokens 5.9 us, of them 2 the launch and 2 the code of scores too close for f32, met for the first
// time.  Instantiated in moe_router_groups.cu (f32 logits) and moe_router_groups_bf16.cu, so that they compile side by side.
#pragma once

#include "moe_router.cuh"

namespace moe {
namespace {

// Eight lanes have a token where no more than eight registers hold it so, else 32.
template <class L>
struct RunGrouped {
    const RouterParams &p;
    bool loss;
    int ctas;
    cudaStream_t s;
    template <int NI, int G, int kGrouped>
    cudaError_t run() const {
        // four kept of a lane's eight and more, whatever k is, to build half as many kernels (32767 x 256 in 8 groups, 8 / 16 / 32 chosen
        // by the largest logit 26.0 / 33.5 / 45.4 us, all kept 27.6 / 36.4 / 50.9; by scores in 16 groups of 16, 8 / 16 chosen 85.6 /
        // 127, all kept 89.3 / 110)
        constexpr int kFew = G == 32 && NI > 4 ? 4 : NI;
        if (loss) return launch(router_kernel<L, NI, G, kFew, true, false, kGrouped>, ctas, kThreads, (size_t)(kWarps + 1) * p.E * 4, 1, s, p);
        return launch(router_kernel<L, NI, G, kFew, false, false, kGrouped>, ctas, kThreads, 0, 1, s, p);
    }
    template <int NI, int G>
    cudaError_t run() const {
        if (NI > 2 && p.each == 1) return run<NI, G, 2>();
        if (NI > 4 && p.each == 2) return run<NI, G, 3>();
        return run<NI, G, 1>();
    }
    cudaError_t run() const {
        const int n = p.groups * p.each;
        if (p.each * 8 >= p.group_size && n <= 8) return n <= 2 ? run<2, 8>() : n <= 4 ? run<4, 8>() : run<8, 8>();
        return n <= 2 ? run<2, 32>() : n <= 4 ? run<4, 32>() : n <= 8 ? run<8, 32>() : n <= 16 ? run<16, 32>() : run<32, 32>();
    }
};

}  // namespace
}  // namespace moe
