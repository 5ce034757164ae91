// moe_fp8_quant.cu -- E4M3 codes with f32 scales of tokens, of SwiGLU's output and gradient, and of weights (definitions in
// include/moe.h).
//
// One pass: a CTA takes tiles of 128 columns by 128 rows (32 where only rows of few tokens are scaled), every value is read once,
// held in registers in f32, and written with the scale of its row's group, of its column's group, or of both.  A warp has whole
// rows of the tile, so a row's largest value is one reduction over the warp; a column's are joined over the warps in shared
// memory.  What bounds it is latency, of loads, reductions and barriers on 15 warps an SM (128 registers each), not a unit: 4096 x 7168
// bf16 both ways 26.3 us, 4.5 TB/s (17.3 at the copy rate), with 58% of the issue slots, 41% of the integer pipe and 36% of the
// memory's rate in use; the columns alone, without the reductions, 16.7.
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
    uint32_t tiles;
};

// Four neighbouring elements as they are in memory.
template <class S>
struct Raw4;
template <>
struct Raw4<float> {
    uint4 r;
    __device__ __forceinline__ void load(const float *p) { r = ld_stream16(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    }
};
template <>
struct Raw4<bf16> {
    uint2 r;
    __device__ __forceinline__ void load(const bf16 *p) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { r = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xFFFF0000u);
        v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xFFFF0000u);
    }
};
// A warp's rows of a tile, `rows` of them (zeros else).
template <class S, int RW>
__device__ __forceinline__ void load_rows(Raw4<S> (&v)[RW], const S *at, int64_t ld, int rows) {
    if (rows == RW) {
#pragma unroll
        for (int r = 0; r < RW; ++r, at += ld) v[r].load(at);
    } else {
#pragma unroll
        for (int r = 0; r < RW; ++r, at += ld) {
            v[r].zero();
            if (r < rows) v[r].load(at);
        }
    }
}

// A group's factor as one number: 1 / sf, or where values are brought up by 2^64 first, minus 1 / (2^64 sf).
__device__ __forceinline__ float factor_of(const GroupScale &g) { return g.up == 1.0f ? g.inv : -g.inv; }
__device__ __forceinline__ float scaled(float v, float f) { return f < 0.0f ? v * 0x1p64f * -f : v * f; }
// The codes of four neighbours under factors of their own, or (`plain`) none of which is negative.
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], float4 f, bool plain) {
    if (plain) {
        const float2 a = __fmul2_rn(make_float2(v[0], v[1]), make_float2(f.x, f.y)), b = __fmul2_rn(make_float2(v[2], v[3]), make_float2(f.z, f.w));
        return e4m3x2(a.x, a.y) | e4m3x2(b.x, b.y) << 16;
    }
    return e4m3x2(scaled(v[0], f.x), scaled(v[1], f.y)) | e4m3x2(scaled(v[2], f.z), scaled(v[3], f.w)) << 16;
}
__device__ __forceinline__ float most(const float (&v)[4]) {
    return fmaxf(fmaxf(fmaxf(fmaxf(0.0f, fabsf(v[0])), fabsf(v[1])), fabsf(v[2])), fabsf(v[3]));
}

// Codes of a warp's rows to `tile` + `at` (its first row's four columns of this lane), W bytes apart, `rows` of them (lanes past the
// last column none).  `factor` may ask other lanes, so the whole warp takes the same way and only the stores are a lane's own.
template <int RW, class F>
__device__ __forceinline__ void put_codes(uint8_t *tile, uint32_t at, uint32_t W, const float (&v)[RW][4], int rows, bool plain, F factor) {
    if (plain && __all_sync(kAll, rows == RW)) {   // almost always: no question asked for a row
#pragma unroll
        for (int r = 0; r < RW; ++r, at += W) *reinterpret_cast<uint32_t *>(tile + at) = codes4(v[r], factor(r), true);
        return;
    }
#pragma unroll
    for (int r = 0; r < RW; ++r, at += W) {
        const float4 f = factor(r);
        if (r < rows) *reinterpret_cast<uint32_t *>(tile + at) = codes4(v[r], f, plain);
    }
}

// A tile's values (RW rows of four columns) with the scales of their groups.
template <int RW, int kWarps>
__device__ __forceinline__ void write_tile(const float (&v)[RW][4], const QuantParams &p, int W, int64_t r0, int c0, int rows, bool blocks,
                                           float (*maxima)[128], float (*factor)[4], float (*row_max)[RW]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = r0 + warp * RW;
    const int groups = (W + 127) / 128;
    const uint32_t at = (uint32_t)(warp * RW) * W + c0 + 4 * lane;   // within the tile's rows
    const bool by_cols = p.col_codes || blocks;
    if (by_cols) {   // first, so that the warps that join the columns need not wait for the rows
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < RW; r += 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = fmaxf(fmaxf(m[i], fabsf(v[r][i])), fabsf(v[r + 1][i]));
        *reinterpret_cast<float4 *>(&maxima[warp][4 * lane]) = make_float4(m[0], m[1], m[2], m[3]);
    }
    if (p.codes && !blocks) {
        // the rows' maxima through shared memory to a lane each (by a select a row the integer pipe, which bounds this, has two more)
        float *mine = row_max[warp];
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const uint32_t all = __reduce_max_sync(kAll, __float_as_uint(most(v[r])));
            if (lane == 0) mine[r] = __uint_as_float(all);
        }
        __syncwarp();
        const GroupScale g = group_scale(lane < RW ? mine[lane] : 0.0f);
        if (lane < RW && row0 + lane < p.T) p.sf[(row0 + lane) * groups + c0 / 128] = g.sf;
        const float own = factor_of(g);
        put_codes(p.codes + r0 * W, at, W, v, rows, !__any_sync(kAll, own < 0.0f), [&](int r) {
            const float f = __shfl_sync(kAll, own, r);
            return make_float4(f, f, f, f);
        });
    }
    if (!by_cols) return;
    __syncthreads();
    if (threadIdx.x < 128) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w += 2) m = fmaxf(fmaxf(m, maxima[w][threadIdx.x]), maxima[w + 1][threadIdx.x]);
        if (blocks) {   // each of the four warps joins 32 columns
            m = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(m)));
            if (lane == 0) factor[0][warp] = m;
        } else {
            const GroupScale g = group_scale(m);
            factor[threadIdx.x / 4][threadIdx.x % 4] = factor_of(g);
            if (c0 % p.H + (int)threadIdx.x < p.H) p.col_sf[r0 / 128 * W + c0 + threadIdx.x] = g.sf;
        }
    }
    __syncthreads();
    float4 f = *reinterpret_cast<const float4 *>(factor[blocks ? 0 : lane]);
    if (blocks) {
        const GroupScale g = group_scale(fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)));
        f.x = f.y = f.z = f.w = factor_of(g);
        if (threadIdx.x == 0) p.sf[r0 / 128 * groups + c0 / 128] = g.sf;
    }
    put_codes((blocks ? p.codes : p.col_codes) + r0 * W, at, W, v, rows,
              !__any_sync(kAll, fminf(fminf(f.x, f.y), fminf(f.z, f.w)) < 0.0f), [&](int) { return f; });
}

// SwiGLU of a row's gate and up columns, or (kGrad) its gradient in their places.
template <int kKind, bool kClamp>
__device__ __forceinline__ void swiglu4(float (&a)[4], float (&u)[4], const float (&d)[4], float clamp) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float g = kClamp ? clamp_of(a[i], clamp) : a[i], up = kClamp ? clamp_of(u[i], clamp) : u[i], s = sigmoid_of(g);
        if (kKind == kSwiglu) {
            a[i] = g * s * up;
        } else {   // da = d u s (1 + g (1 - s)), du = d g s, none through a clamp
            const float da = d[i] * up * (s * fmaf(g, 1.0f - s, 1.0f)), du = d[i] * (g * s);
            a[i] = kClamp && fabsf(a[i]) > clamp ? 0.0f : da;
            u[i] = kClamp && fabsf(u[i]) > clamp ? 0.0f : du;
        }
    }
}

template <class S, int kKind, int RW, int kWarps, int kCtas>
__global__ void __launch_bounds__(kWarps * 32, kCtas) quant_kernel(const __grid_constant__ QuantParams p) {
    constexpr bool kGlu = kKind == kSwiglu || kKind == kGrad;
    constexpr bool kAhead = !kGlu && sizeof(S) == 2;   // registers for the next tile's rows too
    __shared__ alignas(16) float maxima[kKind == kGrad ? 2 : 1][kWarps][128], factor[kKind == kGrad ? 2 : 1][32][4], row_max[kWarps][RW];
    launch_next();
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = (p.H + 127) / 128;
    const uint32_t total = p.tiles;
    const S *v = static_cast<const S *>(p.v), *d = static_cast<const S *>(p.d);
    // a tile's first row and column, and how many of the warp's rows there are (none past the last column)
    auto place = [&](uint32_t tile, int64_t &r0, int &c0, int &rows) {
        const uint32_t tr = tile / across;
        c0 = (int)(tile - tr * across) * 128;
        r0 = (int64_t)tr * (RW * kWarps);
        rows = c0 + 4 * lane < p.H ? (int)max((int64_t)0, min((int64_t)RW, p.T - r0 - warp * RW)) : 0;
    };
    int64_t r0;
    int c0, rows;
    place(blockIdx.x, r0, c0, rows);
    Raw4<S> raw[RW];
    if (kAhead) load_rows<S, RW>(raw, v + (r0 + warp * RW) * p.ld_v + c0 + 4 * lane, p.ld_v, rows);
    for (uint32_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        float a[RW][4];
        if constexpr (kAhead) {
#pragma unroll
            for (int r = 0; r < RW; ++r) raw[r].get(a[r]);
            const int64_t r1 = r0;
            const int c1 = c0, rows1 = rows;
            if (tile + gridDim.x < total) {   // the next tile's while this one is worked on
                place(tile + gridDim.x, r0, c0, rows);
                load_rows<S, RW>(raw, v + (r0 + warp * RW) * p.ld_v + c0 + 4 * lane, p.ld_v, rows);
            }
            write_tile<RW, kWarps>(a, p, p.H, r1, c1, rows1, kKind == kBlocks, maxima[0], factor[0], row_max);
        } else if constexpr (!kGlu) {
            place(tile, r0, c0, rows);
            load_rows<S, RW>(raw, v + (r0 + warp * RW) * p.ld_v + c0 + 4 * lane, p.ld_v, rows);
#pragma unroll
            for (int r = 0; r < RW; ++r) raw[r].get(a[r]);
            write_tile<RW, kWarps>(a, p, p.H, r0, c0, rows, kKind == kBlocks, maxima[0], factor[0], row_max);
        } else {
            place(tile, r0, c0, rows);
            float u[RW][4], e[kKind == kGrad ? RW : 1][4];
            const S *from = v + (r0 + warp * RW) * p.ld_v + c0 + 4 * lane;
            Raw4<S> up[RW], grad[kKind == kGrad ? RW : 1];
            load_rows<S, RW>(raw, from, p.ld_v, rows);
            load_rows<S, RW>(up, from + p.H, p.ld_v, rows);
            if constexpr (kKind == kGrad) load_rows<S, RW>(grad, d + (r0 + warp * RW) * p.ld_d + c0 + 4 * lane, p.ld_d, rows);
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                raw[r].get(a[r]);
                up[r].get(u[r]);
                if constexpr (kKind == kGrad) grad[r].get(e[r]);
            }
            if (p.clamp < INFINITY) {
#pragma unroll
                for (int r = 0; r < RW; ++r) swiglu4<kKind, true>(a[r], u[r], e[kKind == kGrad ? r : 0], p.clamp);
            } else {
#pragma unroll
                for (int r = 0; r < RW; ++r) swiglu4<kKind, false>(a[r], u[r], e[kKind == kGrad ? r : 0], p.clamp);
            }
            write_tile<RW, kWarps>(a, p, kKind == kGrad ? 2 * p.H : p.H, r0, c0, rows, false, maxima[0], factor[0], row_max);
            if constexpr (kKind == kGrad) write_tile<RW, kWarps>(u, p, 2 * p.H, r0, p.H + c0, rows, false, maxima[1], factor[1], row_max);
        }
    }
}

template <class S, int kKind, int RW, int kWarps, int kCtas>
int launch_quant(QuantParams p, cudaStream_t s) {
    const int64_t tiles = ((int64_t)p.T + RW * kWarps - 1) / (RW * kWarps) * ((p.H + 127) / 128);
    if (tiles > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
    p.tiles = (uint32_t)tiles;
    const int dev = this_device(), sms = dev < 0 ? 0 : sm_count(dev);
    if (!sms) return MOE_ERR_CUDA;
    // what the SMs hold at once; each walks on, its next tile on the way
    const unsigned ctas = (unsigned)std::min<int64_t>(tiles, (int64_t)kCtas * sms);
    return launch(quant_kernel<S, kKind, RW, kWarps, kCtas>, ctas, kWarps * 32, 0, 1, s, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
template <class S>
int run(const QuantParams &p, int kind, cudaStream_t s) {
    // Rows and warps of a tile, CTAs an SM.  bf16 tiles of 128 rows in eight warps leave registers for the next tile's rows (4096 x
    // 7168 both ways 26.3 us, columns alone 16.7, rows alone 18.5; without them 29.0, 22.5, 21.8); f32 ones do not (29 both ways,
    // spilled 79).  Rows alone of few tokens in tiles of 32, so that more SMs have one; 1024 rows and more in larger ones (bf16,
    // in tiles of 32 / of 128 rows: 256 x 7168 3.0 / 3.1 us, 512 x 7168 4.8 / 4.1, 1024 x 2048 3.1 / 3.4, 1024 x 7168 7.0 / 6.7, 2048 x
    // 2048 5.0 / 4.2, 2048 x 7168 12.3 / 10.0; f32, 32 / 64 rows: 256 x 7168 3.4 / 3.6, 2048 x 7168 14.4 / 13.2).
    // SwiGLU's gradient holds three inputs: 32 warps of four rows (1777 x 2048 16.9 us, 16 of eight 22).
    constexpr int RW = sizeof(S) == 2 ? 16 : 8, kWarps = 128 / RW;
    if (kind == kBlocks) return launch_quant<S, kBlocks, RW, kWarps, 2>(p, s);
    if (!p.col_codes) {
        if (kind == kPlain && p.T >= 1024) return launch_quant<S, kPlain, RW, 8, sizeof(S) == 2 ? 2 : 4>(p, s);
        return kind == kPlain    ? launch_quant<S, kPlain, 4, 8, 4>(p, s)
               : kind == kSwiglu ? launch_quant<S, kSwiglu, 4, 8, 4>(p, s)
                                 : launch_quant<S, kGrad, 4, 8, 2>(p, s);
    }
    if (kind == kPlain) return launch_quant<S, kPlain, RW, kWarps, 2>(p, s);
    return kind == kSwiglu ? launch_quant<S, kSwiglu, 8, 16, 2>(p, s) : launch_quant<S, kGrad, 4, 32, 1>(p, s);
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
