// moe_linear.cu -- products of a few tokens with FP4 weights (E2M1 codes under
// UE8M0 scales per 32), with the SwiGLU of a gate/up pair or an added input in
// the epilogue.
//
//   y[m, n] = sum over groups q of 2^(s[n, q] - 127) * sum_{k in q} e2m1(w[n, k]) x[m, k]
//
// What bounds it is reading the weights once (half a byte each, 1/16 more for
// scales); what competes is turning codes into operands.  So the codes go
// through one conversion (two codes to two halves per instruction) straight
// into the A fragments of m16n8k16 MMAs whose N is the tokens: the products
// of up to 8 tokens cost the issue slots of one.  E2M1 is exact in f16.
//
// x is nearly always exact too: every 128-column block of a token is scaled by
// the power of two that brings its largest element into [2^14, 2^15), where f16
// keeps all 8 bits of a bf16 down to 2^-31 of that power of two (2^-17; below,
// the error is at most 2^-39 of it, half of f16's smallest step, far under the
// f32 sum's own unless the large element meets a zero weight).  Each CTA
// converts its x once into shared memory, in the order of the B fragments.
//
// Every scale group is summed by itself (two MMAs from zero) and joined in
// f32 under its scale.  Scales are held relative to their row's largest, so
// that no partial sum leaves the f32 range that the result stays in; the
// row's exponent multiplies the finished sum.
//
// Layout (written once by moe_fp4_linear_transform_weights): tiles of 32 rows
// in two halves of 16 (SWIGLU: 8 gate rows and their 8 up rows each), per tile
// and 128-column block 2 KB of codes in fragment order -- lane (g, t) of a
// warp reads for row g, then for row g + 8 of a half, 16 bytes: word t of each
// of the block's four scale groups -- and 128 bytes of scales.  A word holds 8
// consecutive columns, so the fragments of a group use columns in an order of
// their own, the same for codes and x.  Codes and scales of a block lie
// together (2176 bytes): one stream per warp, and tiles of a power of two of
// columns do not start on the same few memory partitions (with 64 KB between
// tiles the 28672 x 4096 product read at 3.5 TB/s).
//
// Measured: 4096 x 7168 with SwiGLU for one token 5.7 us (2.7 TB/s; the bytes
// alone 2.3 us, a product of 75 x 96 takes 3.3), 7168 x 2048 for 5 tokens
// 4.8 us, 28672 x 4096 for 16 tokens 20.9 us (3.1 TB/s; bytes 9.7): there every
// CTA reads and converts all of x (5 to 6 us), and half of the issue slots of
// the rest go to conversions, MMAs and scale products, which wait on one
// another: 6 tiles at 2 warps each give 12 of the 16 warps work.  Simple
// kernels: 165, 160 and 3093 us.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxM = MOE_FP4_LINEAR_MAX_TOKENS;
constexpr int kTileRows = 32;
constexpr int kBlockCodes = 2048;               // bytes of a tile's 128-column block: codes,
constexpr int kBlockBytes = kBlockCodes + 128;  // then scales
constexpr int kMaxDepth = 6;                    // blocks in flight per warp
constexpr int kSumShift = 18;      // partial sums are held times 2^-18: |x| up to the bf16 maximum cannot overflow them
constexpr size_t kMaxSmem = 227 * 1024;

struct LinearParams {
    const bf16 *x;
    int64_t ld_x;
    const uint8_t *blocks_at;
    const int32_t *row_exp;
    const void *add;
    int64_t ld_add;
    void *y;
    int64_t ld_y;
    int M, K, n_out, tiles, blocks;   // blocks: 128-column blocks of a row
    int split, groups;                // CTAs of a cluster that split K; clusters, which share the tiles
    int wk;                           // warps of a CTA that split its part of K for one tile
    bool one_round;                   // every warp has one tile at most
    int depth;                        // blocks in flight per warp: 2, 3, 4 or 6
    float clamp;
    bool x_vec;
};

// 8 codes -> 4 pairs of halves (byte i of w -> h[i], low nibble in the low half).
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// c = A B (the first of a scale group's two), c += A B
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(byte q of s - 127), q known at compile time
__device__ __forceinline__ float group_scale(uint32_t s, int q) {
    return __uint_as_float((q < 3 ? s << (23 - 8 * q) : s >> 1) & 0x7F800000u);
}

// v in [-c, c]; a NaN stays one (minimum and maximum would make it a bound)
__device__ __forceinline__ float clamped(float v, float c) { return v > c ? c : v < -c ? -c : v; }

__device__ __forceinline__ void add4(float4 &a, const float4 &b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// Waits until at most depth - 1 of the warp's groups of copies are under way.
__device__ __forceinline__ void wait_block(int depth) {
    if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else asm volatile("cp.async.wait_group 5;" ::: "memory");
    __syncwarp();   // the scales were copied by other lanes
}

template <class O, bool kSwiglu, int NT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    launch_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    constexpr int kParts = 2 * NT;   // accumulator fragments of a tile: row half u, token group n at 2 n + u
    const int M = p.M;
    const int rank = kCluster ? (int)(blockIdx.x % p.split) : 0;   // clusters are consecutive CTAs
    const int group = kCluster ? (int)(blockIdx.x / p.split) : (int)blockIdx.x;
    const int cta_b0 = kCluster ? p.blocks * rank / p.split : 0;
    const int cta_blocks = (kCluster ? p.blocks * (rank + 1) / p.split : p.blocks) - cta_b0;
    const int max_blocks = kCluster ? (p.blocks + p.split - 1) / p.split : p.blocks;   // the same layout in every CTA
    // smem: the warps' slots, x as halves [block][group][token][t] 16 bytes, the blocks' powers of two [block][16], sums
    const int ring = p.depth * kBlockBytes;
    uint8_t *slots = smem + warp * ring;
    uint4 *xs = reinterpret_cast<uint4 *>(smem + kWarps * ring);
    float *xe = reinterpret_cast<float *>(xs + max_blocks * 16 * M);
    float4 *joined = reinterpret_cast<float4 *>(xe + max_blocks * kMaxM);   // [other rank][tile][part][32], in the first CTA
    float4 *red = joined + (p.split - 1) * (kWarps / p.wk) * kParts * 32;

    const int wn = warp / p.wk, wk = warp % p.wk, tiles_at_once = kWarps / p.wk;
    const int my_tiles = (p.tiles - group + p.groups - 1) / p.groups;
    const int rounds = (my_tiles + tiles_at_once - 1) / tiles_at_once;
    // a lone round leaves the slots free for the join
    const int red_step = p.one_round ? ring / 16 : kParts * 32;
    if (p.one_round) red = reinterpret_cast<float4 *>(smem);
    const int kb0 = cta_blocks * wk / p.wk, nkb = cta_blocks * (wk + 1) / p.wk - kb0;   // within the CTA's part

    // The warp's blocks, round by round, run through its slots by asynchronous copies: a lane copies what it will read
    // itself, so that its own wait is all that is needed.
    const int64_t tile_blocks = (int64_t)p.groups * tiles_at_once * p.blocks;   // from a warp's tile to its next one
    int64_t in_at = ((int64_t)(group + wn * p.groups)) * p.blocks + cta_b0 + kb0;   // block of the next copy
    int in_left = nkb, in_i = wn;
    const uint32_t slot0 = smem_u32(slots), slot_end = slot0 + ring;
    uint32_t in_slot = slot0;
    const uint8_t *source = p.blocks_at + lane * 16;
    auto copy_next = [&]() {
        if (in_left > 0 && in_i < my_tiles) {
            const uint8_t *c = source + in_at * kBlockBytes;
            asm volatile(
                "cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%0 + 512], [%1 + 512], 16;\n\t"
                "cp.async.cg.shared.global [%0 + 1024], [%1 + 1024], 16;\n\t"
                "cp.async.cg.shared.global [%0 + 1536], [%1 + 1536], 16;" ::"r"(in_slot + lane * 16),
                "l"(c)
                : "memory");
            if (lane < 8)
                asm volatile("cp.async.cg.shared.global [%0 + 2048], [%1 + 2048], 16;" ::"r"(in_slot + lane * 16), "l"(c)
                             : "memory");
            ++in_at;
            if (--in_left == 0) in_at += tile_blocks - nkb, in_left = nkb, in_i += tiles_at_once;
            in_slot += kBlockBytes;
            if (in_slot == slot_end) in_slot = slot0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // x -> halves: a half-warp takes one token's block at a time, kBatch items' loads together.  The first ones are asked
    // for before the weights, which would otherwise keep them waiting (a microsecond of a one-token call).
    constexpr int kBatch = NT == 2 ? 16 : 4;
    const int sub = lane & 15, items = cta_blocks * M, item0 = warp * 2 + (lane >> 4);
    const unsigned half = lane < 16 ? 0x0000FFFFu : 0xFFFF0000u;   // the halves may end at different items
    const float inv_m = 1.0f / (float)M;
    uint4 v[kBatch];
    auto block_of = [&](int item) { return (int)(((float)item + 0.5f) * inv_m); };   // item / M: far from rounding
    auto load_x = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int item = i0 + i * 2 * kWarps;
            v[i] = make_uint4(0, 0, 0, 0);
            if (item >= items) continue;
            const int b = block_of(item), k = (cta_b0 + b) * 128 + sub * 8;
            if (k >= p.K) continue;   // K is a multiple of 32: all eight columns are there or none
            const bf16 *src = p.x + (item - b * M) * p.ld_x + k;
            if (p.x_vec) {
                v[i] = ld_stream16(src);
            } else {
                const uint16_t *e = reinterpret_cast<const uint16_t *>(src);
                v[i] = make_uint4((uint32_t)e[0] | (uint32_t)e[1] << 16, (uint32_t)e[2] | (uint32_t)e[3] << 16,
                                  (uint32_t)e[4] | (uint32_t)e[5] << 16, (uint32_t)e[6] | (uint32_t)e[7] << 16);
            }
        }
    };
    auto convert_x = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int item = i0 + i * 2 * kWarps;
            if (item >= items) break;
            const int b = block_of(item), m = item - b * M;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
            top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
            for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
            const int e = max((int)(top >> 7), 33);   // the largest exponent; 33 keeps 2^(e-141-18) a normal float
            const float down = __uint_as_float((uint32_t)(268 - e) << 23);   // 2^(141 - e)
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __fmul2_rn(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), pair(down));
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(f.y), "f"(f.x));
            }
            xs[((b * 4 + (sub >> 2)) * M + m) * 4 + (sub & 3)] = make_uint4(h[0], h[1], h[2], h[3]);
            if (sub == 0) xe[b * kMaxM + m] = __uint_as_float((uint32_t)(e - 14 - kSumShift) << 23);
        }
    };
    wait_for_previous();
    load_x(item0);
#pragma unroll 1
    for (int d = 0; d < p.depth; ++d) copy_next();
    convert_x(item0);
    for (int i0 = item0 + kBatch * 2 * kWarps; i0 < items; i0 += kBatch * 2 * kWarps) {
        load_x(i0);
        convert_x(i0);
    }
    // every CTA of a cluster has started before another one writes to its shared memory
    if (kCluster) cooperative_groups::this_cluster().sync();
    else __syncthreads();

    int row[NT];   // the token whose x this lane loads as column g (tokens past M repeat the last one)
#pragma unroll
    for (int n = 0; n < NT; ++n) row[n] = min(g + 8 * n, M - 1) * 4 + t;

    int out_slot = 0;
    for (int r = 0; r < rounds; ++r) {
        float4 acc[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int i_tile = r * tiles_at_once + wn;
        int row_e[2][2] = {};   // exponents of rows g, g + 8 of the halves, for the end of the round
        if (i_tile < my_tiles) {
            const int32_t *e = p.row_exp + (group + i_tile * p.groups) * kTileRows + g;
            row_e[0][0] = e[0], row_e[0][1] = e[8], row_e[1][0] = e[16], row_e[1][1] = e[24];
#pragma unroll 1
            for (int j = 0; j < nkb; ++j) {
                wait_block(p.depth);
                const uint8_t *slot = slots + out_slot;
                out_slot = out_slot + kBlockBytes == ring ? 0 : out_slot + kBlockBytes;
                uint32_t w[4][4];   // rows g, g + 8 of the halves; their words of the four groups
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(slot + 512 * i + lane * 16);
                    w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
                }
                const uint4 scv = *reinterpret_cast<const uint4 *>(slot + kBlockCodes + g * 16);
                const uint32_t sc[4] = {scv.x, scv.y, scv.z, scv.w};
                float2 sum[kParts][2];   // rows g and g + 8, two tokens each
#pragma unroll
                for (int i = 0; i < kParts; ++i) sum[i][0] = sum[i][1] = make_float2(0.0f, 0.0f);
                const uint4 *xb = xs + (kb0 + j) * 16 * M;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 xv[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xv[n] = xb[q * M * 4 + row[n]];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a[4], c[4];
                        e2m1x8(w[2 * u][q], a);
                        e2m1x8(w[2 * u + 1][q], c);
                        const float s0 = group_scale(sc[2 * u], q), s1 = group_scale(sc[2 * u + 1], q);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float f[4];
                            mma_f16_first(f, a[0], c[0], a[1], c[1], xv[n].x, xv[n].y);
                            mma_f16(f, a[2], c[2], a[3], c[3], xv[n].z, xv[n].w);
                            float2(&sm)[2] = sum[2 * n + u];
                            sm[0] = __ffma2_rn(pair(s0), make_float2(f[0], f[1]), sm[0]);
                            sm[1] = __ffma2_rn(pair(s1), make_float2(f[2], f[3]), sm[1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 e = *reinterpret_cast<const float2 *>(xe + (kb0 + j) * kMaxM + 8 * n + 2 * t);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float4 &v = acc[2 * n + u];
                        const float2 lo = __ffma2_rn(e, sum[2 * n + u][0], make_float2(v.x, v.y));
                        const float2 hi = __ffma2_rn(e, sum[2 * n + u][1], make_float2(v.z, v.w));
                        v = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
                __syncwarp();   // every lane has read the scales
                copy_next();    // into the slot just read
            }
        }
        if (p.wk > 1) {
#pragma unroll
            for (int i = 0; i < kParts; ++i) red[warp * red_step + i * 32 + lane] = acc[i];
            __syncthreads();
        }
        // part i of a tile is finished by the tile's warp i % wk
        if (p.wk > 1 && i_tile < my_tiles) {
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                if (i % p.wk != wk) continue;
                acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int w = 0; w < p.wk; ++w) add4(acc[i], red[(wn * p.wk + w) * red_step + i * 32 + lane]);
            }
        }
        if (kCluster) {
            namespace cg = cooperative_groups;
            cg::cluster_group cluster = cg::this_cluster();
            if (rank > 0 && i_tile < my_tiles) {
                float4 *dst = cluster.map_shared_rank(joined, 0);
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    if (i % p.wk == wk) dst[(((rank - 1) * tiles_at_once + wn) * kParts + i) * 32 + lane] = acc[i];
            }
            cluster.sync();
            if (rank == 0 && i_tile < my_tiles) {
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    if (i % p.wk != wk) continue;
                    for (int o = 0; o < p.split - 1; ++o) add4(acc[i], joined[((o * tiles_at_once + wn) * kParts + i) * 32 + lane]);
                }
            }
        }
        if (i_tile < my_tiles && rank == 0) {
            const int tile = group + i_tile * p.groups;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                if (part % p.wk != wk) continue;
                const int u = part & 1, n = part >> 1, first = tile * kTileRows + 16 * u;
                float v[4] = {acc[part].x, acc[part].y, acc[part].z, acc[part].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // times 2^(exponent + kSumShift), in two steps that are floats
                    const int e = row_e[u][i >> 1] + kSumShift, e1 = e >> 1;
                    v[i] = v[i] * pow2(e1) * pow2(e - e1);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 8 * n + 2 * t + (i & 1);
                    const int col = kSwiglu ? first / 2 + g : first + g + 8 * (i >> 1);
                    if (m >= M || col >= p.n_out || (kSwiglu && i > 1)) continue;
                    float o = v[i];
                    if (kSwiglu) {
                        const float gt = clamped(o, p.clamp), up = clamped(v[(i + 2) & 3], p.clamp);
                        o = gt / (1.0f + expf(-gt)) * up;
                    }
                    if (p.add) o += to_f32(static_cast<const O *>(p.add)[m * p.ld_add + col]);
                    static_cast<O *>(p.y)[m * p.ld_y + col] = from_f32<O>(o);
                }
            }
        }
        // the next round writes `red` and `joined` again, and no CTA leaves while another may still write to it
        if (kCluster) cooperative_groups::this_cluster().sync();
        else if (p.wk > 1 && !p.one_round) __syncthreads();
    }
}

// Row that slot r (0..31) of a tile holds, or -1.
__device__ __forceinline__ int row_of(int tile, int r, int N, bool swiglu) {
    const int n = swiglu ? N / 2 : N;
    const int i = swiglu ? tile * (kTileRows / 2) + (r >> 4) * 8 + (r & 7) : tile * kTileRows + r;
    if (i >= n) return -1;
    return swiglu && (r & 8) ? n + i : i;
}

// One warp per (tile, slot): the row's largest scale, its scales relative to that one, its codes in fragment order.
__global__ void linear_transform_kernel(const uint8_t *w, const uint8_t *w_sf, int N, int K, bool swiglu, int tiles, int blocks,
                                        uint8_t *out, int32_t *row_exp) {
    const int lane = threadIdx.x & 31;
    const int slot = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int tile = slot / kTileRows, r = slot % kTileRows;
    if (tile >= tiles) return;
    const int row = row_of(tile, r, N, swiglu), groups = K / 32;
    int top = 0;
    if (row >= 0)
        for (int q = lane; q < groups; q += 32) top = max(top, (int)w_sf[(int64_t)row * groups + q]);
    top = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)top);
    if (lane == 0) row_exp[slot] = top - 127;
    for (int i = lane; i < blocks * 4; i += 32) {   // group i of the row
        const int64_t at = (int64_t)tile * blocks + (i >> 2);
        const bool in = row >= 0 && i < groups;
        // [block][g][rows g, g + 8, g + 16, g + 24][4 groups]; a scale 2^-127 or less of the largest one counts as 0
        out[at * kBlockBytes + kBlockCodes + (r & 7) * 16 + (r >> 3) * 4 + (i & 3)] =
            in ? (uint8_t)max(0, 127 + (int)w_sf[(int64_t)row * groups + i] - top) : 0;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(w + (int64_t)row * (K / 2)) + i * 4;
        uint32_t *dst = reinterpret_cast<uint32_t *>(out + at * kBlockBytes + (r >> 3) * 512 + (r & 7) * 64);
        for (int t = 0; t < 4; ++t) dst[t * 4 + (i & 3)] = in ? src[t] : 0u;
    }
}

bool valid(const moe_fp4_linear_config *c) {
    if (!c || c->in_features < 32 || c->in_features % 32 || c->in_features > MOE_FP4_LINEAR_MAX_IN) return false;
    if (c->out_features < 1) return false;
    if (c->act != MOE_ACT_NONE && c->act != MOE_ACT_SWIGLU) return false;
    if (c->act == MOE_ACT_SWIGLU && c->out_features % 2) return false;
    return valid_dtype(c->out_dtype) && !isnan(c->act_clamp) && c->act_clamp > 0.0f;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct Layout {
    int tiles, blocks;
    size_t row_exp, total;   // offset; the blocks are at 0
};
Layout layout(const moe_fp4_linear_config *c) {
    Layout l;
    l.tiles = (c->out_features - 1) / kTileRows + 1;   // of gate and up rows alike
    l.blocks = (c->in_features + 127) / 128;
    l.row_exp = up256((size_t)l.tiles * l.blocks * kBlockBytes);
    l.total = l.row_exp + up256((size_t)l.tiles * kTileRows * 4);
    return l;
}

// Shared memory of a CTA that holds `blocks` blocks of x.
size_t smem_bytes(int blocks, int M, int split, int tiles_at_once, int depth, bool join) {
    const int parts = M > 8 ? 4 : 2;
    return (size_t)kWarps * depth * kBlockBytes + (size_t)blocks * (256 * M + 4 * kMaxM) +
           (size_t)((join ? kThreads : 0) + (split - 1) * tiles_at_once * 32) * parts * 16;
}

template <class O, bool kSwiglu, int NT, bool kCluster>
cudaError_t launch_linear(const LinearParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint32_t> done{0};
    const cudaError_t e = smem_limit_once((const void *)linear_kernel<O, kSwiglu, NT, kCluster>, kMaxSmem, done);
    if (e != cudaSuccess) return e;
    return launch(linear_kernel<O, kSwiglu, NT, kCluster>, p.groups * p.split, kThreads, smem, kCluster ? p.split : 1, s, p);
}
template <class O, bool kSwiglu>
cudaError_t launch_linear(const LinearParams &p, size_t smem, cudaStream_t s) {
    if (p.M > 8) return p.split > 1 ? launch_linear<O, kSwiglu, 2, true>(p, smem, s) : launch_linear<O, kSwiglu, 2, false>(p, smem, s);
    return p.split > 1 ? launch_linear<O, kSwiglu, 1, true>(p, smem, s) : launch_linear<O, kSwiglu, 1, false>(p, smem, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_fp4_linear_weight_bytes(const moe_fp4_linear_config *cfg) { return valid(cfg) ? layout(cfg).total : 0; }

int moe_fp4_linear_transform_weights(const moe_fp4_linear_config *cfg, const void *w, const void *w_sf,
                                     void *d_weights, void *stream) {
    if (!valid(cfg) || !w || !w_sf || !d_weights || !aligned_to(w, 16) || !aligned_to(d_weights, 256))
        return MOE_ERR_INVALID_ARG;
    const Layout l = layout(cfg);
    uint8_t *d = static_cast<uint8_t *>(d_weights);
    linear_transform_kernel<<<l.tiles * (kTileRows / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t *>(w), static_cast<const uint8_t *>(w_sf), cfg->out_features, cfg->in_features,
        cfg->act == MOE_ACT_SWIGLU, l.tiles, l.blocks, d, reinterpret_cast<int32_t *>(d + l.row_exp));
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_fp4_linear_forward(const moe_fp4_linear_config *cfg, int num_tokens, const void *x, int64_t ld_x,
                           const void *d_weights, const void *add, int64_t ld_add, void *y, int64_t ld_y,
                           void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens > kMaxM) return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOE_OK;
    const bool swiglu = cfg->act == MOE_ACT_SWIGLU;
    const int n_out = swiglu ? cfg->out_features / 2 : cfg->out_features;
    const size_t os = dtype_bytes(cfg->out_dtype);
    if (!x || !d_weights || !y || ld_x < cfg->in_features || ld_y < n_out || (add && ld_add < n_out))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 2) || !aligned_to(d_weights, 256) || !aligned_to(add, os) || !aligned_to(y, os))
        return MOE_ERR_INVALID_ARG;
    const Layout l = layout(cfg);
    constexpr int sms = 152;
    const uint8_t *wt = static_cast<const uint8_t *>(d_weights);
    LinearParams p;
    p.x = static_cast<const bf16 *>(x);
    p.ld_x = ld_x;
    p.blocks_at = wt;
    p.row_exp = reinterpret_cast<const int32_t *>(wt + l.row_exp);
    p.add = add;
    p.ld_add = ld_add;
    p.y = y;
    p.ld_y = ld_y;
    p.M = num_tokens;
    p.K = cfg->in_features;
    p.n_out = n_out;
    p.tiles = l.tiles;
    p.blocks = l.blocks;
    // K over the CTAs of a cluster (split) and the warps of a CTA (wk): the fewest blocks one after the other on a warp,
    // among what fits in shared memory.  A join of warps counts as one block more, one of CTAs as two (2048 x 16384 for 4
    // tokens: 9.8 us over clusters, 13.6 without; 4096 x 7168 for one token: 5.7 without, 8.5 over pairs).
    size_t smem = 0;
    int best = 1 << 30;
    p.depth = 0;
    for (int split = 1; split <= 8; split *= 2) {
        const int groups = std::min(std::max(1, sms / split), l.tiles);
        const int per_cta = (l.tiles + groups - 1) / groups, blocks = (l.blocks + split - 1) / split;
        for (int wk = 1; wk <= kWarps; wk *= 2) {
            const int rounds = (per_cta * wk + kWarps - 1) / kWarps;
            const int cost = rounds * ((blocks + wk - 1) / wk + (wk > 1) + 2 * (split > 1));
            if (cost >= best) continue;
            for (int d : {kMaxDepth, 4, 3, 2}) {
                const size_t need = smem_bytes(blocks, num_tokens, split, kWarps / wk, d, wk > 1 && rounds > 1);
                if (need > kMaxSmem) continue;
                best = cost, smem = need;
                p.split = split, p.groups = groups, p.wk = wk, p.one_round = rounds == 1, p.depth = d;
                break;
            }
        }
    }
    if (p.depth == 0) return MOE_ERR_UNSUPPORTED;   // no such size within MOE_FP4_LINEAR_MAX_IN
    p.clamp = cfg->act_clamp;
    p.x_vec = aligned_to(x, 16) && ld_x % 8 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = cfg->out_dtype == MOE_DTYPE_F32;
    const cudaError_t e = swiglu ? (f32 ? launch_linear<float, true>(p, smem, s) : launch_linear<bf16, true>(p, smem, s))
                                 : (f32 ? launch_linear<float, false>(p, smem, s) : launch_linear<bf16, false>(p, smem, s));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
