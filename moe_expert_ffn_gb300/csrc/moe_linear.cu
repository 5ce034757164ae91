// moe_linear.cu -- products of a few tokens with FP4 weights (E2M1 codes under
// UE8M0 scales per 32), with the SwiGLU of a gate/up pair or an added input in
// the epilogue.
//
// One warp per output column; a lane takes whole scale groups of 32.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxM = MOE_FP4_LINEAR_MAX_TOKENS;

struct LinearParams {
    const bf16 *x;
    int64_t ld_x;
    const uint8_t *w, *w_sf;
    const void *add;
    int64_t ld_add;
    void *y;
    int64_t ld_y;
    int M, N, K, n_out;
    float clamp;
};

__device__ __forceinline__ float e2m1(uint32_t nib) {
    const float mag = (nib & 6) ? ldexpf(1.0f + 0.5f * (nib & 1), (int)((nib >> 1) & 3) - 1) : 0.5f * (nib & 1);
    return (nib & 8) ? -mag : mag;
}

__device__ __forceinline__ void dot_row(const LinearParams &p, int n, int lane, float (&acc)[kMaxM]) {
#pragma unroll
    for (int m = 0; m < kMaxM; ++m) acc[m] = 0.0f;
    for (int g = lane; g < p.K / 32; g += 32) {
        const float s = ldexpf(1.0f, (int)p.w_sf[(int64_t)n * (p.K / 32) + g] - 127);
        const uint8_t *w = p.w + (int64_t)n * (p.K / 2) + g * 16;
        // the scale multiplies the group's sum: a scaled weight may pass the f32 range where the product does not
        float part[kMaxM];
#pragma unroll
        for (int m = 0; m < kMaxM; ++m) part[m] = 0.0f;
        for (int b = 0; b < 16; ++b) {
            const float w0 = e2m1(w[b] & 15), w1 = e2m1(w[b] >> 4);
#pragma unroll
            for (int m = 0; m < kMaxM; ++m)
                if (m < p.M) {
                    const bf16 *x = p.x + m * p.ld_x + g * 32 + 2 * b;
                    part[m] = fmaf(w0, to_f32(x[0]), fmaf(w1, to_f32(x[1]), part[m]));
                }
        }
#pragma unroll
        for (int m = 0; m < kMaxM; ++m) acc[m] = fmaf(s, part[m], acc[m]);
    }
#pragma unroll
    for (int m = 0; m < kMaxM; ++m) acc[m] = warp_sum(acc[m]);
}

template <class O, bool kSwiglu>
__global__ void __launch_bounds__(kThreads) linear_kernel(const LinearParams p) {
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= p.n_out) return;
    float a[kMaxM], b[kMaxM];
    dot_row(p, n, lane, a);
    if (kSwiglu) dot_row(p, n + p.n_out, lane, b);
#pragma unroll
    for (int m = 0; m < kMaxM; ++m) {
        if (m >= p.M || lane != 0) continue;
        float v = a[m];
        if (kSwiglu) {
            const float g = fminf(fmaxf(a[m], -p.clamp), p.clamp), u = fminf(fmaxf(b[m], -p.clamp), p.clamp);
            v = g / (1.0f + expf(-g)) * u;
        }
        if (p.add) v += to_f32(static_cast<const O *>(p.add)[m * p.ld_add + n]);
        static_cast<O *>(p.y)[m * p.ld_y + n] = from_f32<O>(v);
    }
}

bool valid(const moe_fp4_linear_config *c) {
    if (!c || c->in_features < 32 || c->in_features % 32 || c->out_features < 1) return false;
    if (c->act != MOE_ACT_NONE && c->act != MOE_ACT_SWIGLU) return false;
    if (c->act == MOE_ACT_SWIGLU && c->out_features % 2) return false;
    return valid_dtype(c->out_dtype) && !isnan(c->act_clamp) && c->act_clamp > 0.0f;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }
size_t code_bytes(const moe_fp4_linear_config *c) { return (size_t)c->out_features * (c->in_features / 2); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_fp4_linear_weight_bytes(const moe_fp4_linear_config *cfg) {
    if (!valid(cfg)) return 0;
    return up256(code_bytes(cfg)) + up256((size_t)cfg->out_features * (cfg->in_features / 32));
}

int moe_fp4_linear_transform_weights(const moe_fp4_linear_config *cfg, const void *w, const void *w_sf,
                                     void *d_weights, void *stream) {
    if (!valid(cfg) || !w || !w_sf || !d_weights || !aligned_to(w, 16) || !aligned_to(d_weights, 256))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *d = static_cast<uint8_t *>(d_weights);
    if (cudaMemcpyAsync(d, w, code_bytes(cfg), cudaMemcpyDeviceToDevice, s) != cudaSuccess ||
        cudaMemcpyAsync(d + up256(code_bytes(cfg)), w_sf, (size_t)cfg->out_features * (cfg->in_features / 32),
                        cudaMemcpyDeviceToDevice, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

int moe_fp4_linear_forward(const moe_fp4_linear_config *cfg, int num_tokens, const void *x, int64_t ld_x,
                           const void *d_weights, const void *add, int64_t ld_add, void *y, int64_t ld_y,
                           void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens > kMaxM) return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOE_OK;
    const int n_out = cfg->act == MOE_ACT_SWIGLU ? cfg->out_features / 2 : cfg->out_features;
    const size_t os = dtype_bytes(cfg->out_dtype);
    if (!x || !d_weights || !y || ld_x < cfg->in_features || ld_y < n_out || (add && ld_add < n_out))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 2) || !aligned_to(d_weights, 256) || !aligned_to(add, os) || !aligned_to(y, os))
        return MOE_ERR_INVALID_ARG;
    const uint8_t *wt = static_cast<const uint8_t *>(d_weights);
    LinearParams p{static_cast<const bf16 *>(x), ld_x, wt, wt + up256(code_bytes(cfg)), add, ld_add, y, ld_y,
                   num_tokens, cfg->out_features, cfg->in_features, n_out, cfg->act_clamp};
    const int ctas = (n_out + kThreads / 32 - 1) / (kThreads / 32);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = cfg->out_dtype == MOE_DTYPE_F32;
    if (cfg->act == MOE_ACT_SWIGLU) {
        if (f32) linear_kernel<float, true><<<ctas, kThreads, 0, s>>>(p);
        else linear_kernel<bf16, true><<<ctas, kThreads, 0, s>>>(p);
    } else {
        if (f32) linear_kernel<float, false><<<ctas, kThreads, 0, s>>>(p);
        else linear_kernel<bf16, false><<<ctas, kThreads, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
