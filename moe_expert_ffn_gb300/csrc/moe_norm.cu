// moe_norm.cu -- the norms after one block and before the next, fused with the
// gate, the residual sum and the expert layer's input quantisation, forward
// and backward (formulas in include/moe.h).
//
// One CTA per row holds the row's sum z in shared memory in f32 between the
// two norms, so every input is read once and every output written once.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 304;   // rows of partial column sums in the backward workspace

struct NormFwd {
    moe_norm_io io;
    int T, H, quant;
    float eps, residual_scale;
};

template <class S, class P, int kGate>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormFwd p) {
    extern __shared__ float z[];
    __shared__ float red[2][kWarps];
    const int H = p.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const S *res = static_cast<const S *>(p.io.residual) + t * p.io.ld_residual;
    const P *w_pre = static_cast<const P *>(p.io.w_pre);
    float s2 = 0.0f;
    if (p.io.y) {
        const S *y = static_cast<const S *>(p.io.y) + t * p.io.ld_y;
        S *h = static_cast<S *>(p.io.h) + t * p.io.ld_h;
        const P *w_post = static_cast<const P *>(p.io.w_post);
        const P *gate = static_cast<const P *>(p.io.gate);
        float r1 = 1.0f;
        if (w_post) {
            float s1 = 0.0f;
            for (int i = tid; i < H; i += kThreads) {
                const float v = to_f32(y[i]);
                s1 += v * v;
            }
            s1 = block_sum<kWarps>(s1, red[0]);
            r1 = 1.0f / sqrtf(s1 / (float)H + p.eps);
            if (tid == 0 && p.io.rstd_post) p.io.rstd_post[t] = r1;
        }
        const float gt = kGate == MOE_GATE_TOKEN ? to_f32(gate[t]) : 1.0f;
        for (int i = tid; i < H; i += kThreads) {
            float u = to_f32(y[i]);
            if (w_post) u *= r1 * to_f32(w_post[i]);
            const float g = kGate == MOE_GATE_CHANNEL ? to_f32(gate[i]) : gt;
            const float v = fmaf(g, u, p.residual_scale * to_f32(res[i]));
            z[i] = v;
            h[i] = from_f32<S>(v);
            s2 += v * v;
        }
    } else {
        for (int i = tid; i < H; i += kThreads) {
            const float v = to_f32(res[i]);
            z[i] = v;
            s2 += v * v;
        }
    }
    if (!w_pre) return;
    s2 = block_sum<kWarps>(s2, red[1]);   // also orders the writes of z before the reads below
    const float r2 = 1.0f / sqrtf(s2 / (float)H + p.eps);
    if (tid == 0 && p.io.rstd_pre) p.io.rstd_pre[t] = r2;
    S *n = p.io.n ? static_cast<S *>(p.io.n) + t * p.io.ld_n : nullptr;
    // a warp takes 128 columns at a time, 32 per step
    for (int c = warp * 128; c < H; c += kWarps * 128) {
        float v[4], top = 0.0f, amax[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = c + 32 * j + lane;
            v[j] = i < H ? z[i] * r2 * to_f32(w_pre[i]) : 0.0f;
            if (n && i < H) n[i] = from_f32<S>(v[j]);
            amax[j] = warp_max(fabsf(v[j]));
            top = fmaxf(top, amax[j]);
        }
        if (p.quant == MOE_QUANT_NONE) continue;
        uint8_t *codes = p.io.codes + t * H;
        if (p.quant == MOE_QUANT_FP8_128) {
            const Fp8Scale q = fp8_scale(top);
#pragma unroll
            for (int j = 0; j < 4; ++j) codes[c + 32 * j + lane] = e4m3x2(q.apply(v[j]), 0.0f) & 0xFF;
            if (lane == 0) static_cast<float *>(p.io.sf)[t * (H / 128) + c / 128] = q.sf;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c + 32 * j >= H) break;
                const int e = ue8m0_exponent(amax[j]);
                codes[c + 32 * j + lane] = e4m3x2(scale_down(v[j], e), 0.0f) & 0xFF;
                if (lane == 0) static_cast<uint8_t *>(p.io.sf)[t * (H / 32) + c / 32 + j] = (uint8_t)(e + 127);
            }
        }
    }
}

struct NormBwd {
    moe_norm_grad_io io;
    float *part;   // [parts][3][H]: dw_post, dgate (channel), dw_pre
    int T, H;
    float residual_scale;
};

template <class S, class P, int kGate>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormBwd p) {
    extern __shared__ float D[];
    __shared__ float red[3][kWarps];
    const int H = p.H, tid = threadIdx.x;
    float *a_post = p.part + (int64_t)blockIdx.x * 3 * H, *a_gate = a_post + H, *a_pre = a_post + 2 * H;
    for (int i = tid; i < H; i += kThreads) a_post[i] = a_gate[i] = a_pre[i] = 0.0f;
    const P *w_post = static_cast<const P *>(p.io.w_post);
    const P *w_pre = static_cast<const P *>(p.io.w_pre);
    const P *gate = static_cast<const P *>(p.io.gate);
    const float inv_h = 1.0f / (float)H;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {   // every thread keeps its own columns throughout
        const S *h = static_cast<const S *>(p.io.h) + t * p.io.ld_h;
        const S *dh = p.io.dh ? static_cast<const S *>(p.io.dh) + t * p.io.ld_dh : nullptr;
        const S *dn = p.io.dn ? static_cast<const S *>(p.io.dn) + t * p.io.ld_dn : nullptr;
        const S *y = p.io.y ? static_cast<const S *>(p.io.y) + t * p.io.ld_y : nullptr;
        S *dres = static_cast<S *>(p.io.dresidual) + t * p.io.ld_dresidual;
        float r2 = 0.0f, m2 = 0.0f;
        if (dn) {
            r2 = p.io.rstd_pre[t];
            for (int i = tid; i < H; i += kThreads) m2 += to_f32(dn[i]) * to_f32(w_pre[i]) * (to_f32(h[i]) * r2);
            m2 = block_sum<kWarps>(m2, red[0]) * inv_h;
        }
        const float r1 = w_post ? p.io.rstd_post[t] : 1.0f;
        const float gt = kGate == MOE_GATE_TOKEN ? to_f32(gate[t]) : 1.0f;
        float m1 = 0.0f, sg = 0.0f;
        for (int i = tid; i < H; i += kThreads) {
            float d = dh ? to_f32(dh[i]) : 0.0f;
            if (dn) {
                const float hat = to_f32(h[i]) * r2, g = to_f32(dn[i]);
                a_pre[i] += g * hat;
                d += r2 * (g * to_f32(w_pre[i]) - hat * m2);
            }
            D[i] = d;
            if (!y) continue;
            const float hat = to_f32(y[i]) * r1, w = w_post ? to_f32(w_post[i]) : 1.0f;
            const float gi = kGate == MOE_GATE_CHANNEL ? to_f32(gate[i]) : gt;
            const float du = d * hat * w;
            if (kGate == MOE_GATE_CHANNEL) a_gate[i] += du;
            sg += du;
            if (w_post) {
                a_post[i] += d * gi * hat;
                m1 += d * gi * w * hat;
            }
        }
        if (w_post) m1 = block_sum<kWarps>(m1, red[1]) * inv_h;
        if (kGate == MOE_GATE_TOKEN) {
            sg = block_sum<kWarps>(sg, red[2]);
            if (tid == 0) p.io.dgate[t] = sg;
        }
        for (int i = tid; i < H; i += kThreads) {
            const float d = D[i];
            dres[i] = from_f32<S>(y ? p.residual_scale * d : d);
            if (!y) continue;
            const float gi = kGate == MOE_GATE_CHANNEL ? to_f32(gate[i]) : gt;
            float out = d * gi;
            if (w_post) {
                const float hat = to_f32(y[i]) * r1;
                out = r1 * (out * to_f32(w_post[i]) - hat * m1);
            }
            static_cast<S *>(p.io.dy)[t * p.io.ld_dy + i] = from_f32<S>(out);
        }
        __syncthreads();   // the next row writes `red` again
    }
}

// Column sums of the partials in row order (the same bits every time).
__global__ void __launch_bounds__(kThreads) norm_bwd_sum_kernel(const float *part, int parts, int H, float *dw_post,
                                                                float *dgate, float *dw_pre) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    float *out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dgate : dw_pre;
    if (!out || i >= H) return;
    float s = 0.0f;
    for (int r = 0; r < parts; ++r) s += part[((int64_t)r * 3 + blockIdx.y) * H + i];
    out[i] = s;
}

bool valid(const moe_norm_config *c) {
    if (!c || c->hidden < 1 || c->hidden > MOE_NORM_MAX_HIDDEN) return false;
    if (!valid_dtype(c->stream_dtype) || !valid_dtype(c->param_dtype)) return false;
    if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_TOKEN) return false;
    if (c->quant < MOE_QUANT_NONE || c->quant > MOE_QUANT_UE8M0_32) return false;
    if (c->quant == MOE_QUANT_FP8_128 && c->hidden % 128) return false;
    if (c->quant == MOE_QUANT_UE8M0_32 && c->hidden % 32) return false;
    return c->eps > 0.0f && isfinite(c->eps) && isfinite(c->residual_scale);
}

// `f` is called with the stream's and the parameters' element types and the gate kind.
template <int kGate, class F>
cudaError_t by_types(const moe_norm_config *c, F f) {
    const bool s32 = c->stream_dtype == MOE_DTYPE_F32, p32 = c->param_dtype == MOE_DTYPE_F32;
    if (s32) return p32 ? f.template run<float, float, kGate>() : f.template run<float, bf16, kGate>();
    return p32 ? f.template run<bf16, float, kGate>() : f.template run<bf16, bf16, kGate>();
}
template <class F>
cudaError_t by_config(const moe_norm_config *c, F f) {
    if (c->gate == MOE_GATE_CHANNEL) return by_types<MOE_GATE_CHANNEL>(c, f);
    if (c->gate == MOE_GATE_TOKEN) return by_types<MOE_GATE_TOKEN>(c, f);
    return by_types<MOE_GATE_NONE>(c, f);
}

struct RunFwd {
    const NormFwd &p;
    cudaStream_t s;
    template <class S, class P, int kGate>
    cudaError_t run() const {
        static std::atomic<uint32_t> done{0};
        const cudaError_t e = smem_limit_once((const void *)norm_fwd_kernel<S, P, kGate>, 4 * MOE_NORM_MAX_HIDDEN, done);
        if (e != cudaSuccess) return e;
        norm_fwd_kernel<S, P, kGate><<<p.T, kThreads, 4 * p.H, s>>>(p);
        return cudaGetLastError();
    }
};

struct RunBwd {
    const NormBwd &p;
    int parts;
    cudaStream_t s;
    template <class S, class P, int kGate>
    cudaError_t run() const {
        static std::atomic<uint32_t> done{0};
        const cudaError_t e = smem_limit_once((const void *)norm_bwd_kernel<S, P, kGate>, 4 * MOE_NORM_MAX_HIDDEN, done);
        if (e != cudaSuccess) return e;
        norm_bwd_kernel<S, P, kGate><<<parts, kThreads, 4 * p.H, s>>>(p);
        return cudaGetLastError();
    }
};

bool ld_ok(const void *p, int64_t ld, int H) { return !p || ld >= H; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_forward(const moe_norm_config *cfg, int num_tokens, const moe_norm_io *io, void *stream) {
    if (!valid(cfg) || !io || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    const int H = cfg->hidden;
    const bool quant = cfg->quant != MOE_QUANT_NONE;
    if (!io->y && (io->w_post || io->gate || io->h || io->rstd_post)) return MOE_ERR_INVALID_ARG;
    if (io->y && ((io->gate != nullptr) != (cfg->gate != MOE_GATE_NONE))) return MOE_ERR_INVALID_ARG;
    if (!io->y && !io->w_pre) return MOE_ERR_INVALID_ARG;
    if (!io->w_post && io->rstd_post) return MOE_ERR_INVALID_ARG;
    if (!io->w_pre && (io->n || io->codes || io->sf || io->rstd_pre)) return MOE_ERR_INVALID_ARG;
    if (!quant && (io->codes || io->sf)) return MOE_ERR_INVALID_ARG;
    if (!io->residual || (io->y && !io->h)) return MOE_ERR_INVALID_ARG;
    if (io->w_pre && quant && (!io->codes || !io->sf)) return MOE_ERR_INVALID_ARG;
    if (io->w_pre && !quant && !io->n) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(cfg->stream_dtype), ps = dtype_bytes(cfg->param_dtype);
    if (!ld_ok(io->residual, io->ld_residual, H) || !ld_ok(io->y, io->ld_y, H) || !ld_ok(io->h, io->ld_h, H) ||
        !ld_ok(io->n, io->ld_n, H))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(io->residual, es) || !aligned_to(io->y, es) || !aligned_to(io->h, es) || !aligned_to(io->n, es) ||
        !aligned_to(io->w_post, ps) || !aligned_to(io->w_pre, ps) || !aligned_to(io->gate, ps) ||
        !aligned_to(io->rstd_post, 4) || !aligned_to(io->rstd_pre, 4) || !aligned_to(io->codes, 16) ||
        !aligned_to(io->sf, 4))
        return MOE_ERR_INVALID_ARG;
    NormFwd p{*io, num_tokens, H, io->w_pre ? cfg->quant : (int)MOE_QUANT_NONE, cfg->eps, cfg->residual_scale};
    moe_norm_config c = *cfg;
    if (!io->y) c.gate = MOE_GATE_NONE;
    return by_config(&c, RunFwd{p, static_cast<cudaStream_t>(stream)}) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_workspace_bytes(const moe_norm_config *cfg, int num_tokens) {
    if (!valid(cfg) || num_tokens < 0) return 0;
    const size_t b = (size_t)std::max(1, std::min(num_tokens, kMaxParts)) * 3 * cfg->hidden * 4;
    return (b + 255) / 256 * 256;
}

int moe_norm_backward(const moe_norm_config *cfg, int num_tokens, const moe_norm_grad_io *io, void *d_workspace,
                      void *stream) {
    if (!valid(cfg) || !io || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const int H = cfg->hidden;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_tokens == 0) {   // empty tensors have no address: only the sums over no tokens are written
        const bool channel = cfg->gate == MOE_GATE_CHANNEL;
        if ((io->dw_post && cudaMemsetAsync(io->dw_post, 0, 4 * (size_t)H, s) != cudaSuccess) ||
            (io->dw_pre && cudaMemsetAsync(io->dw_pre, 0, 4 * (size_t)H, s) != cudaSuccess) ||
            (channel && io->dgate && cudaMemsetAsync(io->dgate, 0, 4 * (size_t)H, s) != cudaSuccess))
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!io->y && (io->w_post || io->gate || io->rstd_post || io->dy || io->dw_post || io->dgate))
        return MOE_ERR_INVALID_ARG;
    if (io->y && ((io->gate != nullptr) != (cfg->gate != MOE_GATE_NONE) || (io->gate != nullptr) != (io->dgate != nullptr)))
        return MOE_ERR_INVALID_ARG;
    if ((io->w_post != nullptr) != (io->dw_post != nullptr) || (io->w_pre != nullptr) != (io->dw_pre != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!io->dresidual || (io->y && !io->dy) || (!io->dh && !io->dn)) return MOE_ERR_INVALID_ARG;
    if ((io->dn != nullptr) != (io->w_pre != nullptr) || (io->w_pre && !io->rstd_pre) ||
        (io->w_post && !io->rstd_post) || (io->dn && !io->h))
        return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(cfg->stream_dtype), ps = dtype_bytes(cfg->param_dtype);
    if (!ld_ok(io->h, io->ld_h, H) || !ld_ok(io->y, io->ld_y, H) || !ld_ok(io->dh, io->ld_dh, H) ||
        !ld_ok(io->dn, io->ld_dn, H) || !ld_ok(io->dresidual, io->ld_dresidual, H) || !ld_ok(io->dy, io->ld_dy, H))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(io->h, es) || !aligned_to(io->y, es) || !aligned_to(io->dh, es) || !aligned_to(io->dn, es) ||
        !aligned_to(io->dresidual, es) || !aligned_to(io->dy, es) || !aligned_to(io->w_post, ps) ||
        !aligned_to(io->w_pre, ps) || !aligned_to(io->gate, ps) || !aligned_to(io->rstd_post, 4) ||
        !aligned_to(io->rstd_pre, 4) || !aligned_to(io->dw_post, 4) || !aligned_to(io->dgate, 4) ||
        !aligned_to(io->dw_pre, 4) || !aligned_to(d_workspace, 256))
        return MOE_ERR_INVALID_ARG;
    const bool channel = io->gate && cfg->gate == MOE_GATE_CHANNEL;
    const bool sums = io->dw_post || io->dw_pre || channel;
    if (!d_workspace) return MOE_ERR_INVALID_ARG;
    const int parts = std::min(num_tokens, kMaxParts);
    NormBwd p{*io, static_cast<float *>(d_workspace), num_tokens, H, cfg->residual_scale};
    moe_norm_config c = *cfg;
    if (!io->y) c.gate = MOE_GATE_NONE;
    if (by_config(&c, RunBwd{p, parts, s}) != cudaSuccess) return MOE_ERR_CUDA;
    if (sums) {
        norm_bwd_sum_kernel<<<dim3((H + kThreads - 1) / kThreads, 3), kThreads, 0, s>>>(
            p.part, parts, H, io->dw_post, channel ? io->dgate : nullptr, io->dw_pre);
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
