// moe_fp8_quant.cu -- E4M3 codes with f32 scales of tokens, of SwiGLU's output and gradient, and of weights (definitions in
// include/moe.h).
//
// One pass: a CTA takes 128 columns of 128 rows (32 where only rows are scaled, so that few tokens fill more SMs), every value
// is read once, held in registers in f32, and written with the scale of its row's group, of its column's group, or of both.  A
// warp has whole rows of the tile, so a row's largest value is one reduction over the warp; a column's are joined over the warps
// in shared memory.
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
enum Kind { kPlain, kSwiglu, kGrad, kBlocks };

struct QuantParams {
    const void *v, *d;            // d: the gradient of SwiGLU's output
    int64_t ld_v, ld_d;
    uint8_t *codes, *col_codes;   // [T, W], W = H or (kGrad) 2H
    float *sf, *col_sf;           // [T, ceil(W/128)], [ceil(T/128), W]; kBlocks: sf [ceil(T/128), ceil(W/128)]
    int T, H;
    float clamp;
};

// Four neighbouring elements.
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const uint4 r = ld_stream16(p);
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void load4(const bf16 *p, float (&v)[4]) {
    uint2 r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xFFFF0000u);
    v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xFFFF0000u);
}

// A tile's values (RW rows of four columns) with the scales of their groups.
template <int RW, int kWarps>
__device__ __forceinline__ void write_tile(const float (&v)[RW][4], const QuantParams &p, int W, int64_t r0, int c0, bool on, bool blocks,
                                           float (*shared)[128]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = c0 + 4 * lane;
    const int64_t row0 = r0 + warp * RW;
    float col_max[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.codes && !blocks) {
        float mine = 0.0f;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const float m = fmaxf(fmaxf(fmaxf(fmaxf(0.0f, fabsf(v[r][0])), fabsf(v[r][1])), fabsf(v[r][2])), fabsf(v[r][3]));
            const float all = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(m)));
            if (lane == r) mine = all;
        }
        const GroupScale g = group_scale(mine);
        const int groups = (W + 127) / 128;
        if (lane < RW && row0 + lane < p.T) p.sf[(row0 + lane) * groups + c0 / 128] = g.sf;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const GroupScale s{0.0f, __shfl_sync(kAll, g.inv, r), __shfl_sync(kAll, g.up, r)};
            if (on && row0 + r < p.T)
                *reinterpret_cast<uint32_t *>(p.codes + (row0 + r) * W + col) = s.codes(v[r][0], v[r][1]) | s.codes(v[r][2], v[r][3]) << 16;
        }
    }
    if (!p.col_codes && !blocks) return;
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) col_max[i] = fmaxf(col_max[i], fabsf(v[r][i]));
    __syncthreads();   // the tile before has read its maxima
    *reinterpret_cast<float4 *>(&shared[warp][4 * lane]) = make_float4(col_max[0], col_max[1], col_max[2], col_max[3]);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float4 m = *reinterpret_cast<const float4 *>(&shared[w][4 * lane]);
        col_max[0] = fmaxf(col_max[0], m.x), col_max[1] = fmaxf(col_max[1], m.y);
        col_max[2] = fmaxf(col_max[2], m.z), col_max[3] = fmaxf(col_max[3], m.w);
    }
    uint8_t *to = p.col_codes;
    GroupScale g[4];
    if (blocks) {
        const float m = fmaxf(fmaxf(col_max[0], col_max[1]), fmaxf(col_max[2], col_max[3]));
        g[0] = g[1] = g[2] = g[3] = group_scale(__uint_as_float(__reduce_max_sync(kAll, __float_as_uint(m))));
        to = p.codes;
        if (threadIdx.x == 0) p.sf[r0 / 128 * ((W + 127) / 128) + c0 / 128] = g[0].sf;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = group_scale(col_max[i]);
        if (warp == 0 && on) *reinterpret_cast<float4 *>(p.col_sf + r0 / 128 * W + col) = make_float4(g[0].sf, g[1].sf, g[2].sf, g[3].sf);
    }
#pragma unroll
    for (int r = 0; r < RW; ++r)
        if (on && row0 + r < p.T) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = v[r][i] * g[i].up * g[i].inv;
            *reinterpret_cast<uint32_t *>(to + (row0 + r) * W + col) = e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16;
        }
}

template <class S, int kKind, int RW, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) quant_kernel(const __grid_constant__ QuantParams p) {
    __shared__ float shared[kWarps][128];
    launch_next();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (p.H + 127) / 128, tc = blockIdx.x % tiles;
    const int64_t r0 = (int64_t)(blockIdx.x / tiles) * (RW * kWarps), row0 = r0 + warp * RW;
    const int c0 = tc * 128, col = c0 + 4 * lane;
    const bool on = col < p.H;
    const S *v = static_cast<const S *>(p.v), *d = static_cast<const S *>(p.d);
    float a[RW][4], u[kKind == kSwiglu || kKind == kGrad ? RW : 1][4], e[kKind == kGrad ? RW : 1][4];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const bool real = on && row0 + r < p.T;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[r][i] = 0.0f;
        if (real) load4(v + (row0 + r) * p.ld_v + col, a[r]);
        if constexpr (kKind == kSwiglu || kKind == kGrad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[r][i] = 0.0f;
            if (real) load4(v + (row0 + r) * p.ld_v + p.H + col, u[r]);
        }
        if constexpr (kKind == kGrad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[r][i] = 0.0f;
            if (real) load4(d + (row0 + r) * p.ld_d + col, e[r]);
        }
    }
    if constexpr (kKind == kSwiglu) {
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = clamp_of(a[r][i], p.clamp);
                a[r][i] = g * sigmoid_of(g) * clamp_of(u[r][i], p.clamp);
            }
    }
    if constexpr (kKind == kGrad) {
        // with s = sigmoid_of(g): da = d u s (1 + g (1 - s)), du = d g s, none through a clamp
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g0 = a[r][i], u0 = u[r][i], g = clamp_of(g0, p.clamp), up = clamp_of(u0, p.clamp), s = sigmoid_of(g);
                a[r][i] = fabsf(g0) > p.clamp ? 0.0f : e[r][i] * up * (s * fmaf(g, 1.0f - s, 1.0f));
                u[r][i] = fabsf(u0) > p.clamp ? 0.0f : e[r][i] * (g * s);
            }
        write_tile<RW, kWarps>(a, p, 2 * p.H, r0, c0, on, false, shared);
        write_tile<RW, kWarps>(u, p, 2 * p.H, r0, p.H + c0, on, false, shared);
    } else {
        write_tile<RW, kWarps>(a, p, p.H, r0, c0, on, kKind == kBlocks, shared);
    }
}

template <class S, int kKind, int RW, int kWarps>
int launch_quant(const QuantParams &p, cudaStream_t s) {
    const int64_t ctas = ((int64_t)p.T + RW * kWarps - 1) / (RW * kWarps) * ((p.H + 127) / 128);
    if (ctas > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
    return launch(quant_kernel<S, kKind, RW, kWarps>, (unsigned)ctas, kWarps * 32, 0, 1, s, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
template <class S>
int run(const QuantParams &p, int kind, cudaStream_t s) {
    if (kind == kBlocks) return launch_quant<S, kBlocks, 16, 8>(p, s);
    if (!p.col_codes)
        return kind == kPlain    ? launch_quant<S, kPlain, 4, 8>(p, s)
               : kind == kSwiglu ? launch_quant<S, kSwiglu, 4, 8>(p, s)
                                 : launch_quant<S, kGrad, 4, 8>(p, s);
    return kind == kPlain    ? launch_quant<S, kPlain, 16, 8>(p, s)
           : kind == kSwiglu ? launch_quant<S, kSwiglu, 8, 16>(p, s)
                             : launch_quant<S, kGrad, 8, 16>(p, s);
}
int run(const QuantParams &p, int kind, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F32 ? run<float>(p, kind, s) : run<bf16>(p, kind, s);
}

constexpr int kMaxColumns = 1 << 20;

bool valid(const moe_fp8_quant_config *c) {
    if (!c || c->columns < 16 || c->columns % 16 || c->columns > kMaxColumns) return false;
    if (c->act != MOE_ACT_NONE && (c->act != MOE_ACT_SWIGLU || c->columns % 128)) return false;
    return valid_dtype(c->dtype) && c->act_clamp > 0.0f;
}

bool rows_ok(const void *p, int64_t ld, int64_t cols, size_t es) {
    return p && aligned_to(p, 16) && ld >= cols && ld * (int64_t)es % 16 == 0;
}

// Either form of output is whole or absent, and one is there.
bool out_ok(const moe_fp8_quant_io *o) {
    if (!o || !o->codes != !o->sf || !o->col_codes != !o->col_sf || (!o->codes && !o->col_codes)) return false;
    return aligned_to(o->codes, 16) && aligned_to(o->col_codes, 16) && aligned_to(o->sf, 4) && aligned_to(o->col_sf, 16);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_fp8_quant(const moe_fp8_quant_config *cfg, int num_tokens, const void *v, int64_t ld_v, const moe_fp8_quant_io *out, void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    if (!out_ok(out)) return MOE_ERR_INVALID_ARG;
    const bool glu = cfg->act == MOE_ACT_SWIGLU;
    if (!rows_ok(v, ld_v, (int64_t)cfg->columns * (glu ? 2 : 1), dtype_bytes(cfg->dtype))) return MOE_ERR_INVALID_ARG;
    const QuantParams p{v, nullptr, ld_v, 0, out->codes, out->col_codes, out->sf, out->col_sf, num_tokens, cfg->columns, cfg->act_clamp};
    return run(p, glu ? kSwiglu : kPlain, cfg->dtype, static_cast<cudaStream_t>(stream));
}

int moe_fp8_quant_backward(const moe_fp8_quant_config *cfg, int num_tokens, const void *d, int64_t ld_d, const void *v, int64_t ld_v,
                           const moe_fp8_quant_io *out, void *stream) {
    if (!valid(cfg) || cfg->act != MOE_ACT_SWIGLU || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    if (!out_ok(out)) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(cfg->dtype);
    if (!rows_ok(v, ld_v, 2 * (int64_t)cfg->columns, es) || !rows_ok(d, ld_d, cfg->columns, es)) return MOE_ERR_INVALID_ARG;
    const QuantParams p{v, d, ld_v, ld_d, out->codes, out->col_codes, out->sf, out->col_sf, num_tokens, cfg->columns, cfg->act_clamp};
    return run(p, kGrad, cfg->dtype, static_cast<cudaStream_t>(stream));
}

int moe_fp8_quant_weights(const moe_fp8_quant_config *cfg, int num_rows, const void *w, int64_t ld_w, uint8_t *codes, float *sf,
                          void *stream) {
    if (!valid(cfg) || cfg->act != MOE_ACT_NONE || num_rows < 0) return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    if (!rows_ok(w, ld_w, cfg->columns, dtype_bytes(cfg->dtype)) || !codes || !sf || !aligned_to(codes, 16) || !aligned_to(sf, 4))
        return MOE_ERR_INVALID_ARG;
    const QuantParams p{w, nullptr, ld_w, 0, codes, nullptr, sf, nullptr, num_rows, cfg->columns, cfg->act_clamp};
    return run(p, kBlocks, cfg->dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
