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
// x is exact too: every 128-column block of a token is scaled by the power of
// two that brings its largest element into [2^14, 2^15), where f16 keeps all 8
// bits of a bf16 down to 2^-33 of that element (below, the error is under
// 2^-39 of it, far under the f32 sum's own).  Each CTA converts its x once
// into shared memory, in the order of the B fragments.
//
// Every scale group is summed by itself (two MMAs from zero) and joined in
// f32 under its scale.  Scales are held relative to their row's largest, so
// that no partial sum leaves the f32 range that the result stays in; the
// row's exponent multiplies the finished sum.
//
// Layout (written once by moe_fp4_linear_transform_weights): tiles of 16 rows
// (SWIGLU: 8 gate rows and their 8 up rows), per tile and 128-column block 1 KB
// of codes in fragment order -- lane (g, t) of a warp loads for row g, then
// for row g + 8, 16 bytes: word t of each of the block's four scale groups --
// and 64 bytes of scales.  A word holds 8 consecutive columns, so the
// fragments of a group use columns in an order of their own, the same for
// codes and x.
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
constexpr int kMaxDepth = 8;       // 128-column blocks in flight per warp
constexpr int kSlotBytes = 1280;   // of one block in shared memory: codes, and every lane's own copy of its scales
constexpr int kBlockCodes = 1024;  // bytes of a tile's 128-column block
constexpr int kBlockScales = 64;
constexpr int kSumShift = 18;      // partial sums are held times 2^-18: |x| up to the bf16 maximum cannot overflow them
constexpr size_t kMaxSmem = 227 * 1024;

struct LinearParams {
    const bf16 *x;
    int64_t ld_x;
    const uint8_t *codes, *scales;
    const int32_t *row_exp;
    const void *add;
    int64_t ld_add;
    void *y;
    int64_t ld_y;
    int M, K, n_out, tiles, blocks;   // blocks: 128-column blocks of a row
    int split, groups;                // CTAs of a cluster that split K; clusters, which share the tiles
    int wk;                           // warps of a CTA that split its part of K for one tile
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

// 2^(byte q of s - 127)
template <int q>
__device__ __forceinline__ float group_scale(uint32_t s) {
    return __uint_as_float((q < 3 ? s << (23 - 8 * q) : s >> 1) & 0x7F800000u);
}

__device__ __forceinline__ void add4(float4 &a, const float4 &b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// Waits until at most kDepth - 1 of this thread's groups of copies are under way.
template <int kDepth>
__device__ __forceinline__ void wait_block() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
}

template <class O, bool kSwiglu, int NT, bool kCluster, int kDepth>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int M = p.M;
    const int rank = kCluster ? (int)(blockIdx.x % p.split) : 0;   // clusters are consecutive CTAs
    const int group = kCluster ? (int)(blockIdx.x / p.split) : (int)blockIdx.x;
    const int cta_b0 = kCluster ? p.blocks * rank / p.split : 0;
    const int cta_blocks = (kCluster ? p.blocks * (rank + 1) / p.split : p.blocks) - cta_b0;
    const int max_blocks = kCluster ? (p.blocks + p.split - 1) / p.split : p.blocks;   // the same layout in every CTA
    // smem: the warps' slots, x as halves [block][group][token][t] 16 bytes, the blocks' powers of two [block][16], sums
    uint8_t *slots = smem + warp * (kDepth * kSlotBytes);
    uint4 *xs = reinterpret_cast<uint4 *>(smem + kWarps * kDepth * kSlotBytes);
    float *xe = reinterpret_cast<float *>(xs + max_blocks * 16 * M);
    float4 *red = reinterpret_cast<float4 *>(xe + max_blocks * kMaxM);
    float4 *joined = red + kThreads * NT;   // [other rank][tile][NT][32], in the cluster's first CTA

    const int wn = warp / p.wk, wk = warp % p.wk, tiles_at_once = kWarps / p.wk;
    const int my_tiles = (p.tiles - group + p.groups - 1) / p.groups;
    const int rounds = (my_tiles + tiles_at_once - 1) / tiles_at_once;
    const int kb0 = cta_blocks * wk / p.wk, nkb = cta_blocks * (wk + 1) / p.wk - kb0;   // within the CTA's part

    // The warp's blocks, round by round, run through its slots by asynchronous copies: a lane copies what it will read
    // itself, so that its own wait is all that is needed.
    const int64_t tile_blocks = (int64_t)p.groups * tiles_at_once * p.blocks;   // from a warp's tile to its next one
    int64_t in_at = ((int64_t)(group + wn * p.groups)) * p.blocks + cta_b0 + kb0;   // block of the next copy
    int in_left = nkb, in_i = wn;
    const uint32_t slot0 = smem_u32(slots), slot_end = slot0 + kDepth * kSlotBytes;
    uint32_t in_slot = slot0;
    const uint8_t *codes = p.codes + lane * 16, *scales = p.scales + g * 8;
    auto copy_next = [&]() {
        if (in_left > 0 && in_i < my_tiles) {
            const uint8_t *c = codes + in_at * kBlockCodes;
            asm volatile(
                "cp.async.cg.shared.global [%0], [%1], 16;\n\tcp.async.cg.shared.global [%0 + 512], [%1 + 512], 16;" ::"r"(
                    in_slot + lane * 16),
                "l"(c)
                : "memory");
            asm volatile("cp.async.ca.shared.global [%0 + 1024], [%1], 8;" ::"r"(in_slot + lane * 8),
                         "l"(scales + in_at * kBlockScales)
                         : "memory");
            ++in_at;
            if (--in_left == 0) in_at += tile_blocks - nkb, in_left = nkb, in_i += tiles_at_once;
            in_slot += kSlotBytes;
            if (in_slot == slot_end) in_slot = slot0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int d = 0; d < kDepth; ++d) copy_next();

    // x -> halves: a half-warp takes one block of every token, four tokens' loads at a time
    {
        const int sub = lane & 15;
        const unsigned half = lane < 16 ? 0x0000FFFFu : 0xFFFF0000u;   // the halves may end at different blocks
        for (int b = warp * 2 + (lane >> 4); b < cta_blocks; b += kWarps * 2) {
            const int k = (cta_b0 + b) * 128 + sub * 8;
            for (int m0 = 0; m0 < M; m0 += 4) {
                uint32_t v[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (m0 + i >= M) break;
                    const bf16 *src = p.x + (m0 + i) * p.ld_x + k;
                    v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
                    if (k >= p.K) continue;   // K is a multiple of 32: all eight columns are there or none
                    if (p.x_vec) {
                        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src));
                        v[i][0] = q.x, v[i][1] = q.y, v[i][2] = q.z, v[i][3] = q.w;
                    } else {
                        const uint16_t *e = reinterpret_cast<const uint16_t *>(src);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[i][j] = (uint32_t)e[2 * j] | (uint32_t)e[2 * j + 1] << 16;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = m0 + i;
                    if (m >= M) break;
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = max(top, max(v[i][j] & 0x7FFFu, (v[i][j] >> 16) & 0x7FFFu));
#pragma unroll
                    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
                    const int e = max((int)(top >> 7), 33);   // the largest exponent; 33 keeps 2^(e-141-18) a normal float
                    const float down = __uint_as_float((uint32_t)(268 - e) << 23);   // 2^(141 - e)
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = __uint_as_float(v[i][j] << 16) * down, c = __uint_as_float(v[i][j] & 0xFFFF0000u) * down;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(c), "f"(a));
                    }
                    xs[((b * 4 + (sub >> 2)) * M + m) * 4 + (sub & 3)] = make_uint4(h[0], h[1], h[2], h[3]);
                    if (sub == 0) xe[b * kMaxM + m] = __uint_as_float((uint32_t)(e - 14 - kSumShift) << 23);
                }
            }
        }
    }
    // every CTA of a cluster has started before another one writes to its shared memory
    if (kCluster) cooperative_groups::this_cluster().sync();
    else __syncthreads();

    int row[NT];   // the token whose x this lane loads as column g (tokens past M repeat the last one)
#pragma unroll
    for (int n = 0; n < NT; ++n) row[n] = min(g + 8 * n, M - 1) * 4 + t;

    int out_slot = 0;
    for (int r = 0; r < rounds; ++r) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        const int i_tile = r * tiles_at_once + wn;
        if (i_tile < my_tiles) {
            {
#pragma unroll 1
                for (int j = 0; j < nkb; ++j) {
                    wait_block<kDepth>();
                    const uint8_t *slot = slots + out_slot;
                    const uint4 lo = *reinterpret_cast<const uint4 *>(slot + lane * 16);
                    const uint4 hi = *reinterpret_cast<const uint4 *>(slot + 512 + lane * 16);
                    const uint2 sc = *reinterpret_cast<const uint2 *>(slot + 1024 + lane * 8);
                    out_slot = out_slot + kSlotBytes == kDepth * kSlotBytes ? 0 : out_slot + kSlotBytes;
                    const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
                    float sum[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[n][i] = 0.0f;
                    const uint4 *xb = xs + (kb0 + j) * 16 * M;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t a[4], c[4];
                        e2m1x8(wl[q], a);
                        e2m1x8(wh[q], c);
                        const float s0 = q == 0   ? group_scale<0>(sc.x)
                                         : q == 1 ? group_scale<1>(sc.x)
                                         : q == 2 ? group_scale<2>(sc.x)
                                                  : group_scale<3>(sc.x);
                        const float s1 = q == 0   ? group_scale<0>(sc.y)
                                         : q == 1 ? group_scale<1>(sc.y)
                                         : q == 2 ? group_scale<2>(sc.y)
                                                  : group_scale<3>(sc.y);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 xv = xb[q * M * 4 + row[n]];
                            float f[4];
                            mma_f16_first(f, a[0], c[0], a[1], c[1], xv.x, xv.y);
                            mma_f16(f, a[2], c[2], a[3], c[3], xv.z, xv.w);
                            sum[n][0] = fmaf(s0, f[0], sum[n][0]);
                            sum[n][1] = fmaf(s0, f[1], sum[n][1]);
                            sum[n][2] = fmaf(s1, f[2], sum[n][2]);
                            sum[n][3] = fmaf(s1, f[3], sum[n][3]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 e = *reinterpret_cast<const float2 *>(xe + (kb0 + j) * kMaxM + 8 * n + 2 * t);
                        acc[n][0] = fmaf(e.x, sum[n][0], acc[n][0]);
                        acc[n][1] = fmaf(e.y, sum[n][1], acc[n][1]);
                        acc[n][2] = fmaf(e.x, sum[n][2], acc[n][2]);
                        acc[n][3] = fmaf(e.y, sum[n][3], acc[n][3]);
                    }
                    copy_next();   // into the slot just read
                }
            }
        }
        if (p.wk > 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                red[(warp * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            __syncthreads();
        }
        // warp n of the tile finishes the tokens of column group n (a lone warp all of them)
        if (p.wk > 1 && i_tile < my_tiles) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (wk != n) continue;
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int w = 0; w < p.wk; ++w) add4(s, red[((wn * p.wk + w) * NT + n) * 32 + lane]);
                acc[n][0] = s.x, acc[n][1] = s.y, acc[n][2] = s.z, acc[n][3] = s.w;
            }
        }
        if (kCluster) {
            namespace cg = cooperative_groups;
            cg::cluster_group cluster = cg::this_cluster();
            if (rank > 0 && i_tile < my_tiles) {
                float4 *dst = cluster.map_shared_rank(joined, 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (p.wk == 1 || wk == n)
                        dst[(((rank - 1) * tiles_at_once + wn) * NT + n) * 32 + lane] =
                            make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            }
            cluster.sync();
            if (rank == 0 && i_tile < my_tiles) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (p.wk > 1 && wk != n) continue;
                    float4 s = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                    for (int o = 0; o < p.split - 1; ++o) add4(s, joined[((o * tiles_at_once + wn) * NT + n) * 32 + lane]);
                    acc[n][0] = s.x, acc[n][1] = s.y, acc[n][2] = s.z, acc[n][3] = s.w;
                }
            }
        }
        if (i_tile < my_tiles && rank == 0) {
            const int tile = group + i_tile * p.groups;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (p.wk > 1 && wk != n) continue;
                const int e0 = p.row_exp[tile * 16 + g], e1 = p.row_exp[tile * 16 + g + 8];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = ldexpf(acc[n][i], (i < 2 ? e0 : e1) + kSumShift);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 8 * n + 2 * t + (i & 1);
                    const int col = kSwiglu ? tile * 8 + g : tile * 16 + g + 8 * (i >> 1);
                    if (m >= M || col >= p.n_out || (kSwiglu && i > 1)) continue;
                    float v = acc[n][i];
                    if (kSwiglu) {
                        const float gt = fminf(fmaxf(v, -p.clamp), p.clamp);
                        const float up = fminf(fmaxf(acc[n][(i + 2) & 3], -p.clamp), p.clamp);
                        v = gt / (1.0f + expf(-gt)) * up;
                    }
                    if (p.add) v += to_f32(static_cast<const O *>(p.add)[m * p.ld_add + col]);
                    static_cast<O *>(p.y)[m * p.ld_y + col] = from_f32<O>(v);
                }
            }
        }
        // the next round writes `red` and `joined` again, and no CTA leaves while another may still write to it
        if (kCluster) cooperative_groups::this_cluster().sync();
        else if (p.wk > 1) __syncthreads();
    }
}

// Row that slot r (0..15) of a tile holds, or -1.
__device__ __forceinline__ int row_of(int tile, int r, int N, bool swiglu) {
    const int n = swiglu ? N / 2 : N;
    const int i = swiglu ? tile * 8 + (r & 7) : tile * 16 + r;
    if (i >= n) return -1;
    return swiglu && r >= 8 ? n + i : i;
}

// One warp per (tile, slot): the row's largest scale, its scales relative to that one, its codes in fragment order.
__global__ void linear_transform_kernel(const uint8_t *w, const uint8_t *w_sf, int N, int K, bool swiglu, int tiles, int blocks,
                                        uint8_t *codes, uint8_t *scales, int32_t *row_exp) {
    const int lane = threadIdx.x & 31;
    const int slot = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int tile = slot >> 4, r = slot & 15;
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
        // [block][g][row half][4 groups]; a scale 2^-127 or less of the largest one counts as 0
        scales[at * kBlockScales + (r & 7) * 8 + (r >> 3) * 4 + (i & 3)] =
            in ? (uint8_t)max(0, 127 + (int)w_sf[(int64_t)row * groups + i] - top) : 0;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(w + (int64_t)row * (K / 2)) + i * 4;
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + at * kBlockCodes + (r >> 3) * 512 + (r & 7) * 64);
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
    size_t scales, row_exp, total;   // offsets; codes are at 0
};
Layout layout(const moe_fp4_linear_config *c) {
    Layout l;
    l.tiles = c->act == MOE_ACT_SWIGLU ? (c->out_features / 2 + 7) / 8 : (c->out_features + 15) / 16;
    l.blocks = (c->in_features + 127) / 128;
    const size_t n = (size_t)l.tiles * l.blocks;
    l.scales = n * kBlockCodes;
    l.row_exp = l.scales + up256(n * kBlockScales);
    l.total = l.row_exp + up256((size_t)l.tiles * 16 * 4);
    return l;
}

// Shared memory of a CTA that holds `blocks` blocks of x.
size_t smem_bytes(int blocks, int M, int split, int tiles_at_once, int depth) {
    const int nt = M > 8 ? 2 : 1;
    return (size_t)kWarps * depth * kSlotBytes + (size_t)blocks * (256 * M + 4 * kMaxM) +
           (size_t)(kThreads + (split - 1) * tiles_at_once * 32) * nt * 16;
}

template <class O, bool kSwiglu, int NT, bool kCluster, int kDepth>
cudaError_t launch(const LinearParams &p, size_t smem, cudaStream_t s) {
    static std::atomic<uint32_t> done{0};
    const cudaError_t e = smem_limit_once((const void *)linear_kernel<O, kSwiglu, NT, kCluster, kDepth>, kMaxSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(p.groups * p.split);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = p.split;
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    c.attrs = a;
    c.numAttrs = kCluster ? 1 : 0;
    return cudaLaunchKernelEx(&c, linear_kernel<O, kSwiglu, NT, kCluster, kDepth>, p);
}
template <class O, bool kSwiglu, int NT, bool kCluster>
cudaError_t launch(const LinearParams &p, size_t smem, int depth, cudaStream_t s) {
    return depth == kMaxDepth ? launch<O, kSwiglu, NT, kCluster, kMaxDepth>(p, smem, s)
                              : launch<O, kSwiglu, NT, kCluster, kMaxDepth / 2>(p, smem, s);
}
template <class O, bool kSwiglu>
cudaError_t launch(const LinearParams &p, size_t smem, int depth, cudaStream_t s) {
    if (p.M > 8)
        return p.split > 1 ? launch<O, kSwiglu, 2, true>(p, smem, depth, s) : launch<O, kSwiglu, 2, false>(p, smem, depth, s);
    return p.split > 1 ? launch<O, kSwiglu, 1, true>(p, smem, depth, s) : launch<O, kSwiglu, 1, false>(p, smem, depth, s);
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
    linear_transform_kernel<<<(l.tiles * 16 + 7) / 8, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t *>(w), static_cast<const uint8_t *>(w_sf), cfg->out_features, cfg->in_features,
        cfg->act == MOE_ACT_SWIGLU, l.tiles, l.blocks, d, d + l.scales, reinterpret_cast<int32_t *>(d + l.row_exp));
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
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    const uint8_t *wt = static_cast<const uint8_t *>(d_weights);
    LinearParams p;
    p.x = static_cast<const bf16 *>(x);
    p.ld_x = ld_x;
    p.codes = wt;
    p.scales = wt + l.scales;
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
    // K is split over a cluster where the tokens' x does not fit one CTA's shared memory, or where there are so few
    // tiles that half the SMs would idle and each part keeps 8 blocks
    size_t smem = 0;
    int depth = kMaxDepth;
    for (p.split = 1;; p.split *= 2) {
        if (p.split > 8) return MOE_ERR_UNSUPPORTED;
        p.groups = std::min(std::max(1, sms / p.split), l.tiles);
        const int per_cta = (l.tiles + p.groups - 1) / p.groups, blocks = (l.blocks + p.split - 1) / p.split;
        // a tile's K over wk warps: the fewest blocks one after the other on a warp, a join counted as one more, among
        // what fits (two warps at least where there are two token groups to finish)
        int best = 1 << 30;
        for (int wk = num_tokens > 8 ? 2 : 1; wk <= kWarps; wk *= 2) {
            const int rounds = (per_cta * wk + kWarps - 1) / kWarps;
            const int cost = rounds * ((blocks + wk - 1) / wk + (wk > 1));
            int d = kMaxDepth;
            size_t need = smem_bytes(blocks, num_tokens, p.split, kWarps / wk, d);
            if (need > kMaxSmem) need = smem_bytes(blocks, num_tokens, p.split, kWarps / wk, d /= 2);
            if (need <= kMaxSmem && cost < best) best = cost, p.wk = wk, depth = d, smem = need;
        }
        if (best == 1 << 30) continue;
        if (p.split < 8 && l.tiles * p.split * 2 <= sms && l.blocks / (p.split * 2) >= 8) continue;
        break;
    }
    p.clamp = cfg->act_clamp;
    p.x_vec = aligned_to(x, 16) && ld_x % 8 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = cfg->out_dtype == MOE_DTYPE_F32;
    const cudaError_t e = swiglu ? (f32 ? launch<float, true>(p, smem, depth, s) : launch<bf16, true>(p, smem, depth, s))
                                 : (f32 ? launch<float, false>(p, smem, depth, s) : launch<bf16, false>(p, smem, depth, s));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
