// moe_fp8_linear.cu -- dense products in E4M3 with f32 scales per 128 (definitions in include/moe.h): the forward product, its
// input's gradient and its weight's gradient.
//
// All three are one product of rows and columns over a contracted axis D, cut into blocks of 128:
//     out[r, c] = sum_b sr(r, b) sc(c, b) sum_{d in b} rows[r, d] cols[c, d]
//   forward        rows = x  [T, K], cols = W [N, K]:  sr per token, sc per 128 columns
//   input's        rows = dy [T, N], cols = W^T:       sr per token, sc per 128 columns
//   weight's       rows = dy^T,      cols = x^T (D = T): sr and sc per row and column
// The transposed operands are not copied: the tensor core reads a tile whose contracted axis is the slower one in shared
// memory as it is ("MN-major"), so every operand is loaded from the layout in which its maker wrote it.
//
// The scales are floats, which the tensor core cannot apply, so each block of 128 has an accumulator of its own in TMEM, read
// and folded into f32 registers while the next ones are computed: out += TMEM * (sr sc), in block order, so the same call gives
// the same bits.
//
// Two kernels.  With many rows, 256 x 256 tiles on CTA pairs (fp8_wide_kernel), bound by the fold: a 256 x 256 x 128 block
// takes the fold warps of an SM some 800 cycles (TMEM reads and their latency, 128 x 256 multiply-adds, the hand-over), the
// tensor cores 512, so they are busy 57% of 2048 x 28672 x 4096 (178 to 190 us, 2.5 to 2.7 PFLOP/s; called for seconds, at the lower
// clock of that load, 196 to 205).  With few, tiles of 128 columns by 16 to 64 rows with the contracted axis split over clusters
// (fp8_small_kernel), bound by the weights' way through one wave of CTAs and what lies around it: launch, first copies, the join
// (4096 x 7168 for one token 8.6 us, of them 4.3 for the weights' bytes).
// plan_for() chooses by what each is estimated to take.
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_gemm_common.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

enum Mode { kForward, kSwiglu, kInput, kWeight };
constexpr bool rows_mn(int m) { return m == kWeight; }                  // whether an operand's contracted axis is the slower one
constexpr bool cols_mn(int m) { return m == kInput || m == kWeight; }

// The status block of every launch: moe_device.cuh's error words.
__device__ int g_status[kErrWords];

struct Fp8Params {
    const float *row_sf, *col_sf;
    int64_t rs_row, rs_blk;       // row_sf[row * rs_row + block * rs_blk]
    int64_t cs_col, cs_blk;       // col_sf[col / 128 (weight's: col) * cs_col + block * cs_blk]
    const void *add;
    int64_t ld_add;
    void *out;                    // f32 or bf16 by `f32`, or codes with `sf`
    int64_t ld_out;
    float *sf;
    int R, C, DB;                 // rows and columns of the output, blocks of the contracted axis
    int tiles_r, tiles_c, split, stages;
    int f32;
    int out_stages;               // stages that a wide tile's output passes through, 0: written directly (codes)
    int wait_us;                  // 0, or (a test of the timeout) the limit of every wait, with CTA 0's first copies withheld
    float clamp;
};

// Waits for a barrier's phase, at most two seconds (or wait_us); false when it or another wait of the CTA gave up.  The clock, the
// limit and the abort flag are looked at every 256 polls, and none of them before.
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, volatile int *abort_flag, const Fp8Params &p) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 255) == 0) {
            if (*abort_flag) return false;
            const uint64_t now = globaltimer_ns(), limit = p.wait_us ? 1000ull * (uint64_t)p.wait_us : kWaitTimeoutNs;
            if (!t0) {
                t0 = now;
            } else if (now - t0 > limit) {
                *abort_flag = 1;
                raise_timeout(g_status);
                return false;
            }
        }
    }
}
// The same whatever the abort flag says: for what is in flight when a CTA ends.
__device__ __forceinline__ void await_end(uint32_t bar, uint32_t parity, const Fp8Params &p) {
    const uint64_t limit = p.wait_us ? 1000ull * (uint64_t)p.wait_us : kWaitTimeoutNs;
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit) return;
}

constexpr uint32_t kPanel = 128 * 128;   // 128 rows or columns of one block
constexpr int kChunk = 8;                // blocks whose scales are brought to shared memory together

// Shared-memory descriptor of 128 rows or columns of a block, 128-byte swizzled, whether the contracted axis is the faster one or the
// slower one: one 128-byte atom across, groups of eight (rows, or contracted elements) 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) { return sw128_kmajor_desc(saddr); }
// What 32 contracted elements add to it.
template <bool kMN>
__device__ constexpr uint32_t operand_step() { return kMN ? 32 * 128 / 16 : 2; }

constexpr uint32_t idesc_major(bool a_mn, bool b_mn) { return (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u); }

__device__ __forceinline__ float swiglu_of(float g, float u, float c) {
    g = clamp_of(g, c);
    return g * sigmoid_of(g) * clamp_of(u, c);
}

// ============================================================================
// Many rows: 256 x 256 tiles on CTA pairs
// ============================================================================
// A pair's MMA reads 128 rows and 128 columns of each CTA's, half of what two single CTAs would read, so the ring's three stages
// hold two blocks each, one barrier for both.  The stores and what is added go through a stage too, by bulk copies beside the
// next tile's blocks (2048 x 28672 x 4096 182 us, weight's gradient with add 140; written and read directly, by all CTAs at once
// at a tile's end, 187 and 174).  Measured besides: 4096 x 4096 x 7168 with SwiGLU and codes 108 us (256 tiles on 76 pairs: 3.4 waves take 4), input's
// gradient 4096 x 7168 x 2048 54 (1.7 waves take 2), weight's 4096 x 4096 x 7168 with add 140 (a scale a column more to multiply
// by, 235 MB of sums read and written).
constexpr int kWideWarps = 12;           // 0 copies, 1 MMA, 2 scales, 4..11 fold and store
constexpr int kWideThreads = 32 * kWideWarps;
constexpr int kFoldWarp0 = 4;
constexpr int kFoldWarps = 8;
constexpr int kWideStages = 3;
constexpr uint32_t kWideStage = 4 * kPanel;   // two blocks of this CTA's 128 rows and of its half of the columns
constexpr int kRowPitch = 132;           // floats between two blocks of row scales: writers of 4 rows x 8 blocks meet no bank twice
// Registers of the four other warps and of the fold warps: 128 x 72 + 256 x 216 threads' are the 384 x 168 of the launch.
constexpr int kOtherRegs = 72, kFoldRegs = 216;
static_assert(128 * kOtherRegs + 256 * kFoldRegs <= kWideThreads * 168, "registers of the launch");
constexpr int kRowGroup = 16;            // row tiles that the walk takes together

struct alignas(8) WideCtrl {
    uint64_t full[kWideStages], empty[kWideStages];
    uint64_t tfull[2], tempty[2];
    uint64_t sfull[2], sempty[2];
    // a stage is the output's (with what is added to it), and holds it; of four tiles in turn, because the three stages may all be
    // granted before the first is written
    uint64_t granted[4][2], written[4][2];
    uint64_t halves[4];              // a row's two fold warps have written their maxima
    uint32_t tmem_base;
    uint32_t where[4][2];            // the granted stage's address (the fold warps have no register for what says it)
    int abort;
    float amax[2][kFoldWarps][32];
};

template <int kMode>
struct WideScales {
    float row[2][kChunk * kRowPitch];
    float col[2][kMode == kWeight ? kChunk * 256 : kChunk * 2];
};

template <int kMode>
constexpr size_t wide_smem() {
    return 1024 + (size_t)kWideStages * kWideStage + sizeof(WideScales<kMode>) + sizeof(WideCtrl);
}

struct WideTile {
    int tr, tc;
};
// Row tiles in groups of 16, in a group all of them for a column tile before the next one: what a wave of tiles reads stays in L2.
__device__ __forceinline__ WideTile wide_tile(int64_t tile, const Fp8Params &p) {
    const int64_t per = (int64_t)kRowGroup * p.tiles_c;
    const int g = (int)(tile / per), first = g * kRowGroup, n = min(kRowGroup, p.tiles_r - first);
    const int local = (int)(tile - g * per);
    return {first + local % n, local / n};
}

// acc += the warp's 2 x 64 TMEM columns times their scales; `release` once the last ones are in registers.
template <bool kCol, class F>
__device__ __forceinline__ void fold_wide(float2 (&acc)[64], uint32_t t0, uint32_t t1, float s0, float s1, uint32_t cs, F release) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float v[16];
        tmem_ld16((c < 4 ? t0 : t1) + 16 * (c & 3), v);
        tmem_ld_wait();
        if (c == 7) release();
        const float2 s = pair(c < 4 ? s0 : s1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = s, g = s;
            if (kCol) {
                const uint4 k = ld_shared16(cs + 64 * c + 16 * i);
                f = __fmul2_rn(s, make_float2(__uint_as_float(k.x), __uint_as_float(k.y)));
                g = __fmul2_rn(s, make_float2(__uint_as_float(k.z), __uint_as_float(k.w)));
            }
            acc[8 * c + 2 * i] = __ffma2_rn(make_float2(v[4 * i], v[4 * i + 1]), f, acc[8 * c + 2 * i]);
            acc[8 * c + 2 * i + 1] = __ffma2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), g, acc[8 * c + 2 * i + 1]);
        }
    }
}

// A tile's output, as 128 rows of 128 bytes ("panels", 128-byte swizzled): its first byte in a row, and how many panels there are.
struct OutTile {
    int x, panels;
};
template <int kMode>
__device__ __forceinline__ OutTile out_tile(const Fp8Params &p, int tc) {
    const int es = p.f32 ? 4 : 2, width = (kMode == kSwiglu ? 128 : 256) * es;
    return {tc * width, min(width, p.C * es - tc * width + 127) / 128};
}

// A thread's outputs to its row of the panels from `panel` on, added to what is there with `add`.
template <int kPairs>
__device__ __forceinline__ void put_row(const float2 (&acc)[64], uint32_t panel, int row, bool f32, bool add) {
    const uint32_t at = panel + row * 128, swz = row & 7;
    if (f32) {
#pragma unroll
        for (int k = 0; k < kPairs / 2; ++k) {
            const uint32_t a = at + (k / 8) * kPanel + (((k & 7) ^ swz) << 4);
            float4 v = make_float4(acc[2 * k].x, acc[2 * k].y, acc[2 * k + 1].x, acc[2 * k + 1].y);
            if (add) {
                const uint4 w = ld_shared16(a);
                v.x += __uint_as_float(w.x), v.y += __uint_as_float(w.y), v.z += __uint_as_float(w.z), v.w += __uint_as_float(w.w);
            }
            st_shared_v4(a, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kPairs / 4; ++k) {
        const uint32_t a = at + (k / 8) * kPanel + (((k & 7) ^ swz) << 4);
        uint32_t w[4] = {0, 0, 0, 0};
        if (add) {
            const uint4 u = ld_shared16(a);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 v = acc[4 * k + i];
            if (add) v.x += __uint_as_float(w[i] << 16), v.y += __uint_as_float(w[i] & 0xFFFF0000u);
            w[i] = bf16x2(v.x, v.y);
        }
        st_shared_v4(a, w[0], w[1], w[2], w[3]);
    }
}

// Asks for a box of a tensor to be brought to L2, where every later write of it shows: for what an earlier kernel may still write.
__device__ __forceinline__ void prefetch_box(const CUtensorMap *tm, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tm), "r"(x), "r"(y) : "memory");
}

// 16 bytes of scales to shared memory, zeros where there are none.
__device__ __forceinline__ void copy_scales(float *to, const float *from, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(on ? 16 : 0) : "memory");
}
// An arrival (one of the barrier's count) when this thread's copies have landed.
__device__ __forceinline__ void arrive_when_copied(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int kMode>
__global__ void __launch_bounds__(kWideThreads, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_cols,
                    const __grid_constant__ CUtensorMap tm_add, const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Fp8Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = align1024(raw);
    uint8_t *after = smem_raw + (base - raw) + kWideStages * kWideStage;
    WideScales<kMode> &sc = *reinterpret_cast<WideScales<kMode> *>(after);
    WideCtrl *ctrl = reinterpret_cast<WideCtrl *>(after + sizeof(WideScales<kMode>));
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31, rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const int DB = p.DB, stages = (DB + 1) / 2;
    const int64_t total = (int64_t)p.tiles_r * p.tiles_c;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_rows);
        tma_prefetch_desc(&tm_cols);
        for (int s = 0; s < kWideStages; ++s) {
            mbar_init(smem_u32(&ctrl->full[s]), 1);
            mbar_init(smem_u32(&ctrl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&ctrl->tfull[b]), 1);
            mbar_init(smem_u32(&ctrl->tempty[b]), 2 * kFoldWarps);
            mbar_init(smem_u32(&ctrl->sfull[b]), kMode == kWeight ? 32 : 1);
            mbar_init(smem_u32(&ctrl->sempty[b]), kFoldWarps);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_u32(&ctrl->granted[i >> 1][i & 1]), 1);
            mbar_init(smem_u32(&ctrl->written[i >> 1][i & 1]), p.out_stages == 2 ? kFoldWarps / 2 : kFoldWarps);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&ctrl->halves[i]), 2);
        ctrl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctrl->tmem_base), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    launch_next();
    const uint32_t tmem = ctrl->tmem_base;
    volatile int *abort_flag = &ctrl->abort;
    const uint32_t full_c = mapa_shared(smem_u32(&ctrl->full[0]), 0), tempty_c = mapa_shared(smem_u32(&ctrl->tempty[0]), 0);
    wait_for_previous();

    if (warp < kFoldWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 0) {
            // ---- copies: each CTA its 128 rows and its half of the columns (SwiGLU: gate rows of W in the even CTA, up rows in the odd)
            const uint64_t pol = policy_evict_normal();
            int it = 0, done = 0;
            bool ok = true;
            for (int64_t tile = cluster; ok && tile < total; tile += clusters, ++done) {
                const WideTile t = wide_tile(tile, p);
                const int r0 = t.tr * 256 + (int)rank * 128;
                const int c0 = kMode == kSwiglu ? t.tc * 128 + (int)rank * p.C : t.tc * 256 + (int)rank * 128;
                for (int ks = 0; ks < stages; ++ks, ++it) {
                    const int s = it % kWideStages, n = min(2, DB - 2 * ks);
                    if (!await(smem_u32(&ctrl->empty[s]), ((it / kWideStages) & 1) ^ 1, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctrl->full[s]), (uint32_t)n * 4 * kPanel);
                        const uint32_t dst = base + s * kWideStage, full = full_c + 8u * s;
                        for (int j = 0; j < n; ++j) {
                            if (p.wait_us && blockIdx.x == 0) break;
                            const int d = (2 * ks + j) * 128;
                            tma_load_2d_pair(dst + j * kPanel, &tm_rows, rows_mn(kMode) ? r0 : d, rows_mn(kMode) ? d : r0, full, pol);
                            tma_load_2d_pair(dst + (2 + j) * kPanel, &tm_cols, cols_mn(kMode) ? c0 : d, cols_mn(kMode) ? d : c0, full,
                                             pol);
                        }
                    }
                    __syncwarp();
                }
                for (int e = 0; ok && e < p.out_stages; ++e, ++it) {   // and the stages of its output
                    const int s = it % kWideStages;
                    if (!await(smem_u32(&ctrl->empty[s]), ((it / kWideStages) & 1) ^ 1, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const OutTile o = out_tile<kMode>(p, t.tc);
                        const int n = p.add ? min(4, o.panels - 4 * e) : 0;
                        const uint32_t granted = smem_u32(&ctrl->granted[done & 3][e]);
                        ctrl->where[done & 3][e] = base + s * kWideStage;
                        if (n > 0) mbar_arrive_expect_tx(granted, (uint32_t)n * kPanel);
                        else mbar_arrive(granted);
                        for (int i = 0; i < n; ++i)
                            tma_load_2d(base + s * kWideStage + i * kPanel, &tm_add, o.x + (4 * e + i) * 128, r0, granted, pol);
                    }
                    __syncwarp();
                }
            }
            for (int i = max(0, it - kWideStages); i < it; ++i)   // the last copies land before the pair ends
                await_end(smem_u32(&ctrl->empty[i % kWideStages]), (i / kWideStages) & 1, p);
        } else if (warp == 1) {
            // ---- MMA (one thread of the even CTA): a stage's first block into accumulator 0, its second into 1
            if (rank == 0 && lane == 0) {
                constexpr uint32_t idesc = idesc_e4m3_f32(256, 256) | idesc_major(rows_mn(kMode), cols_mn(kMode));
                const uint64_t a0 = operand_desc(base), w0 = operand_desc(base + 2 * kPanel);
                int it = 0, last = -1;
                uint32_t ph = 0, tph[2] = {1, 1};   // ph: of each stage
                bool ok = true;
                for (int64_t tile = cluster; ok && tile < total; tile += clusters, it += p.out_stages) {
                    int s = it % kWideStages;
                    for (int ks = 0; ok && ks < stages; ++ks, ++it) {
                        const int n = min(2, DB - 2 * ks);
                        if (!await(smem_u32(&ctrl->full[s]), (ph >> s) & 1, abort_flag, p)) {
                            ok = false;
                            break;
                        }
                        ph ^= 1u << s;
                        const uint64_t a = a0 + s * (kWideStage / 16), w = w0 + s * (kWideStage / 16);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (j >= n) break;
                            if (!await(smem_u32(&ctrl->tempty[j]), tph[j], abort_flag, p)) {
                                ok = false;
                                break;
                            }
                            tph[j] ^= 1;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_pair_e4m3(tmem + j * 256, a + j * (kPanel / 16) + kk * operand_step<rows_mn(kMode)>(),
                                               w + j * (kPanel / 16) + kk * operand_step<cols_mn(kMode)>(), idesc, kk > 0);
                            umma_pair_commit(smem_u32(&ctrl->tfull[j]), 3);
                        }
                        if (ok) umma_pair_commit(smem_u32(&ctrl->empty[s]), 3);
                        last = it;
                        if (++s == kWideStages) s = 0;
                    }
                }
                if (last >= 0) await_end(smem_u32(&ctrl->empty[last % kWideStages]), (last / kWideStages) & 1, p);
            }
        } else if (warp == 2) {
            // ---- scales of eight blocks at a time to shared memory
            int ch = 0;
            bool ok = true;
            for (int64_t tile = cluster; ok && tile < total; tile += clusters) {
                const WideTile t = wide_tile(tile, p);
                const int r0 = t.tr * 256 + (int)rank * 128;
                for (int k0 = 0; k0 < DB; k0 += kChunk, ++ch) {
                    const int slot = ch & 1;
                    if (!await(smem_u32(&ctrl->sempty[slot]), ((ch >> 1) & 1) ^ 1, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    if (kMode == kWeight) {   // neighbouring rows and columns lie together, sizes are multiples of 16
                        const int r = r0 + 4 * (int)lane, c = t.tc * 256 + 4 * (int)lane;
                        const int n = min(kChunk, DB - k0);
                        for (int j = 0; j < n; ++j) {
                            const int64_t b = k0 + j;
                            copy_scales(&sc.row[slot][j * kRowPitch + 4 * lane], p.row_sf + b * p.rs_blk + r, r < p.R);
                            copy_scales(&sc.col[slot][j * 256 + 4 * lane], p.col_sf + b * p.cs_blk + c, c < p.C);
                            copy_scales(&sc.col[slot][j * 256 + 128 + 4 * lane], p.col_sf + b * p.cs_blk + c + 128, c + 128 < p.C);
                        }
                        arrive_when_copied(smem_u32(&ctrl->sfull[slot]));
                    } else {   // eight blocks of a row lie together: a load takes them of four rows
                        const int j = lane & 7, b = k0 + j;
#pragma unroll 8
                        for (int i = 0; i < 32; ++i) {
                            const int r = r0 + (int)(lane >> 3) + 4 * i;
                            sc.row[slot][j * kRowPitch + (lane >> 3) + 4 * i] =
                                b < DB && r < p.R ? p.row_sf[(int64_t)r * p.rs_row + b] : 0.0f;
                        }
                        if (lane < 16) {
                            const int h = lane >> 3;
                            const int cb = kMode == kSwiglu ? t.tc + h * (p.C / 128) : t.tc * 2 + h;
                            const bool on = b < DB && (kMode == kSwiglu || cb * 128 < p.C);
                            sc.col[slot][j * 2 + h] = on ? p.col_sf[cb * p.cs_col + b * p.cs_blk] : 0.0f;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&ctrl->sfull[slot]));
                    }
                }
            }
        } else if (p.out_stages && lane == 0) {
            // ---- stores: the output's stages as the fold warps have written them, given back when they are read
            int it = stages, done = 0;
            bool ok = true;
            for (int64_t tile = cluster; ok && tile < total; tile += clusters, it += stages + p.out_stages, ++done) {
                const WideTile t = wide_tile(tile, p);
                const int r0 = t.tr * 256 + (int)rank * 128;
                const OutTile o = out_tile<kMode>(p, t.tc);
                for (int e = 0; e < p.out_stages; ++e) {
                    const int s = (it + e) % kWideStages;
                    if (!await(smem_u32(&ctrl->written[done & 3][e]), (done >> 2) & 1, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    for (int i = 4 * e; r0 < p.R && i < min(4 * e + 4, o.panels); ++i)
                        tma_store_2d(&tm_out, o.x + i * 128, r0, base + s * kWideStage + (i - 4 * e) * kPanel);
                    tma_store_commit();
                }
                if (!ok) break;
                if (p.out_stages == 2) {
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    mbar_arrive(smem_u32(&ctrl->empty[it % kWideStages]));
                }
                tma_store_wait_read();
                mbar_arrive(smem_u32(&ctrl->empty[(it + p.out_stages - 1) % kWideStages]));
            }
            tma_store_wait_all();
        }
    } else {
        // ---- fold the blocks' accumulators, own 128 rows; warp: 32 rows, half of the columns
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFoldRegs));
        const int q = warp & 3, h = (warp - kFoldWarp0) >> 2;
        const int lrow = q * 32 + (int)lane;
        // SwiGLU: 64 gate columns and the 64 up columns that belong to them
        const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + (kMode == kSwiglu ? 64 * h : 128 * h);
        const uint32_t t1 = t0 + (kMode == kSwiglu ? 128 : 64);
        int ch = 0, done = 0;
        uint32_t phases = 0;
        bool ok = true;
        for (int64_t tile = cluster; ok && tile < total; tile += clusters, ++done) {
            const WideTile t = wide_tile(tile, p);
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
            for (int k0 = 0; ok && k0 < DB; k0 += kChunk, ++ch) {
                const int slot = ch & 1;
                if (!await(smem_u32(&ctrl->sfull[slot]), (ch >> 1) & 1, abort_flag, p)) {
                    ok = false;
                    break;
                }
                const int n = min(kChunk, DB - k0);
                for (int j = 0; j < n; ++j) {
                    const int b = j & 1;
                    const float sr = sc.row[slot][j * kRowPitch + lrow];
                    float s0 = sr, s1 = sr;
                    uint32_t cs = 0;
                    if (kMode == kWeight) {
                        cs = smem_u32(&sc.col[slot][j * 256 + h * 128]);
                    } else if (kMode == kSwiglu) {
                        s0 = sr * sc.col[slot][2 * j], s1 = sr * sc.col[slot][2 * j + 1];
                    } else {
                        s0 = s1 = sr * sc.col[slot][2 * j + h];
                    }
                    if (!await(smem_u32(&ctrl->tfull[b]), (phases >> b) & 1, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    phases ^= 1u << b;
                    tc_fence_after();
                    fold_wide<kMode == kWeight>(acc, t0 + b * 256, t1 + b * 256, s0, s1, cs, [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(tempty_c + 8u * b);
                    });
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctrl->sempty[slot]));
            }
            if (!ok) break;
            const int64_t row = (int64_t)t.tr * 256 + rank * 128 + lrow;
            if (kMode == kSwiglu) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    acc[i].x = swiglu_of(acc[i].x, acc[32 + i].x, p.clamp);
                    acc[i].y = swiglu_of(acc[i].y, acc[32 + i].y, p.clamp);
                    amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
                }
                const int col = t.tc * 128 + h * 64;
                if (p.sf) {
                    // the other 64 columns of the group of 128 are another warp's
                    float (&all)[kFoldWarps][32] = ctrl->amax[done & 1];
                    all[warp - kFoldWarp0][lane] = amax;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctrl->halves[q]));
                    if (!await(smem_u32(&ctrl->halves[q]), done & 1, abort_flag, p)) break;
                    amax = fmaxf(amax, all[(warp - kFoldWarp0) ^ 4][lane]);
                    const GroupScale g = group_scale(amax);
                    if (row < p.R) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = g.codes(acc[2 * i].x, acc[2 * i].y) | g.codes(acc[2 * i + 1].x, acc[2 * i + 1].y) << 16;
                        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + row * p.ld_out + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                        if (h == 0) p.sf[row * (p.C / 128) + t.tc] = g.sf;
                    }
                    continue;
                }
            }
            // through a stage of the ring and a copy from there: the stores, all CTAs' at once, do not hold up the next tile
            const int e = kMode != kSwiglu && p.out_stages == 2 ? h : 0;
            if (!await(smem_u32(&ctrl->granted[done & 3][e]), (done >> 2) & 1, abort_flag, p)) break;
            const uint32_t stage = ctrl->where[done & 3][e];
            const bool f32 = kMode == kWeight || p.f32;
            const int before = kMode == kSwiglu ? (f32 ? 2 : 1) : f32 ? 0 : 2;   // panels of the other half before this one's
            put_row<kMode == kSwiglu ? 32 : 64>(acc, stage + h * before * kPanel, lrow, f32, p.add != nullptr);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctrl->written[done & 3][e]));
        }
    }
    __syncwarp();
    // neither CTA leaves or frees TMEM while the pair's MMA may still touch it
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ============================================================================
// Few rows: tiles of 128 columns x BT rows, the contracted axis split over a cluster
// ============================================================================
constexpr int kSmallThreads = 32 * 12;   // 0 copies, 1 and 2 MMA, 3 scales, 4..11 fold
constexpr int kSmallFold0 = 4;
constexpr int kAhead = 16;               // panels of the weight that a CTA asks for before the kernel before it has ended

constexpr int kMaxStages = 5;
constexpr size_t kSmHalf = 115712, kSmAll = 232448;   // shared memory of a CTA, two and one of them an SM

template <int BT>
constexpr int small_bufs() { return BT <= 64 ? 4 : 2; }
template <int kMode, int BT>
constexpr uint32_t small_stage() { return 2 * kPanel + (kMode == kSwiglu ? 1 : 2) * BT * 128; }
// Whether the cluster's CTAs send one another their sums; those of 128 rows have no room but the stages', and are fetched.
template <int BT, bool kSplit>
constexpr bool small_sends() { return kSplit && BT <= 64; }

template <int kMode, int BT>
struct SmallCtrl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[2][small_bufs<BT>()], tempty[2][small_bufs<BT>()];
    uint64_t sfull[2], sempty[2];
    uint64_t sums;
    uint32_t tmem_base;
    int abort;
    alignas(16) float sc[2][kChunk * (BT + 4)];
    float lane_sc[2][kMode == kWeight ? kChunk * 128 : 4];
};
// Bytes of the sums that a CTA is sent for `rows` rows of a tile: [rank][row of its][set][128].
constexpr size_t sent_bytes(int rows, int split) { return (size_t)((rows + split - 1) / split) * split * 1024; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Four bytes to a CTA of the cluster, counted by a barrier of its.
__device__ __forceinline__ void send(uint32_t to, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to), "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ float4 ld_cluster16(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 plus(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Four consecutive outputs, and of add.
__device__ __forceinline__ float4 load4(const Fp8Params &p, int64_t row, int col) {
    if (p.f32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p.add) + row * p.ld_add + col);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const bf16 *>(p.add) + row * p.ld_add + col);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(const Fp8Params &p, float4 a, int64_t row, int col) {
    if (p.f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * p.ld_out + col) = a;
    else
        *reinterpret_cast<uint2 *>(static_cast<bf16 *>(p.out) + row * p.ld_out + col) = make_uint2(bf16x2(a.x, a.y), bf16x2(a.z, a.w));
}

// act, quantisation, add and store of four columns of a row; a lane has them, a warp 128.
template <bool kGlu>
__device__ __forceinline__ void finish4(const Fp8Params &p, float4 a, float4 u, float4 add, int64_t row, int tc) {
    const int lane = threadIdx.x & 31, col = tc * 128 + 4 * lane;
    if (kGlu) {
        a.x = swiglu_of(a.x, u.x, p.clamp), a.y = swiglu_of(a.y, u.y, p.clamp);
        a.z = swiglu_of(a.z, u.z, p.clamp), a.w = swiglu_of(a.w, u.w, p.clamp);
        if (p.sf) {
            const float mine = fmaxf(fmaxf(fmaxf(fmaxf(0.0f, fabsf(a.x)), fabsf(a.y)), fabsf(a.z)), fabsf(a.w));
            const GroupScale g = group_scale(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mine))));
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.out) + row * p.ld_out + col) = g.codes(a.x, a.y) | g.codes(a.z, a.w) << 16;
            if (lane == 0) p.sf[row * (p.C / 128) + tc] = g.sf;
            return;
        }
    } else {
        a = plus(a, u);
    }
    if (col < p.C) store4(p, plus(a, add), row, col);
}

// Two panels of 128 columns a stage: two neighbouring blocks (SwiGLU: gate and up rows of one), each with an MMA thread,
// accumulators and four fold warps of its own.  TMEM lanes are the output's columns, its columns the rows: the weight is the MMA's
// 128-row operand, so that 16 rows cost 16 columns.  The cluster's CTAs have a part of the contracted axis each and send their
// sums, row by row, to the CTA that joins that row.  Measured: one token's 4096 x 7168 with SwiGLU and codes 8.6 us (with one MMA
// thread for both panels, no weights asked for before the kernel before has ended and sums fetched by who joins them 10.0);
// 128 x 7168 x 2048 8.6 us (2.7 at the copy rate); 16 x 28672 x 4096 21.5 us (5.5 TB/s).
template <int kMode, int BT, bool kSplit>
__global__ void __launch_bounds__(kSmallThreads, BT == 16 ? 2 : 1)
    fp8_small_kernel(const __grid_constant__ CUtensorMap tm_rows, const __grid_constant__ CUtensorMap tm_cols,
                     const __grid_constant__ Fp8Params p) {
    extern __shared__ uint8_t smem_raw[];
    using Ctrl = SmallCtrl<kMode, BT>;
    constexpr int kBufs = small_bufs<BT>();
    const int kStages = p.stages;
    constexpr uint32_t kStage = small_stage<kMode, BT>(), kRows = BT * 128;
    constexpr uint32_t kTmem = 2 * kBufs * BT;
    constexpr bool kGlu = kMode == kSwiglu, kSend = small_sends<BT, kSplit>();
    const uint32_t raw = smem_u32(smem_raw), base = align1024(raw);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem_raw + (base - raw) + kStages * kStage);
    float *sent = reinterpret_cast<float *>(ctrl + 1);
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31, rank = kSplit ? cluster_ctarank() : 0;
    const int split = kSplit ? p.split : 1, tile = blockIdx.x / split, tr = tile % p.tiles_r, tc = tile / p.tiles_r;
    const int r0 = tr * BT, rows = min(BT, p.R - r0);
    const int DB = p.DB, all = kGlu ? DB : (DB + 1) / 2;                   // stages of the whole axis
    const int s0 = (int)((int64_t)all * rank / split), s1 = (int)((int64_t)all * (rank + 1) / split);   // this CTA's

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_rows);
        tma_prefetch_desc(&tm_cols);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctrl->full[s]), 1);
            mbar_init(smem_u32(&ctrl->empty[s]), 2);
        }
        for (int j = 0; j < 2; ++j) {
            for (int b = 0; b < kBufs; ++b) {
                mbar_init(smem_u32(&ctrl->tfull[j][b]), 1);
                mbar_init(smem_u32(&ctrl->tempty[j][b]), 4);
            }
            mbar_init(smem_u32(&ctrl->sfull[j]), kMode == kWeight ? 32 : 1);
            mbar_init(smem_u32(&ctrl->sempty[j]), 8);
        }
        mbar_init(smem_u32(&ctrl->sums), 1);
        ctrl->abort = 0;
        fence_mbar_init();
        // rows rank, rank + split, ... are this CTA's to join: every CTA of the cluster sends it 128 sums of both sets for each
        if (kSend) mbar_arrive_expect_tx(smem_u32(&ctrl->sums), (uint32_t)((max(rows - (int)rank, 0) + split - 1) / split * split * 1024));
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctrl->tmem_base), kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_next();
    if (kSend) cluster_arrive();   // the others may send from here on
    const uint32_t tmem = ctrl->tmem_base;
    volatile int *abort_flag = &ctrl->abort;
    // the weight's part in L2 while the kernel before this one ends
    if (kMode != kWeight && warp == 3) {
        const int panel = 2 * s0 + (int)lane;
        if (lane < kAhead && panel < (kGlu ? 2 * s1 : min(2 * s1, DB))) {
            const int d = (kGlu ? panel >> 1 : panel) * 128, c0 = tc * 128 + (kGlu ? (panel & 1) * p.C : 0);
            prefetch_box(&tm_cols, cols_mn(kMode) ? c0 : d, cols_mn(kMode) ? d : c0);
        }
    }
    wait_for_previous();

    if (warp == 0) {
        const uint64_t pol_w = p.tiles_r > 1 ? policy_evict_normal() : policy_evict_first(), pol_x = policy_evict_last();
        int s = 0;
        uint32_t ph = 1;
        for (int st = s0; st < s1; ++st) {
            const int n = kGlu ? 2 : min(2, DB - 2 * st);
            if (!await(smem_u32(&ctrl->empty[s]), ph, abort_flag, p)) break;
            if (lane == 0) {
                const uint32_t full = smem_u32(&ctrl->full[s]), dst = base + s * kStage;
                mbar_arrive_expect_tx(full, (uint32_t)n * kPanel + (kGlu ? 1 : n) * kRows);
                for (int j = 0; j < n; ++j) {
                    if (p.wait_us && blockIdx.x == 0) break;
                    const int d = (kGlu ? st : 2 * st + j) * 128, c0 = tc * 128 + (kGlu ? j * p.C : 0);
                    tma_load_2d(dst + j * kPanel, &tm_cols, cols_mn(kMode) ? c0 : d, cols_mn(kMode) ? d : c0, full, pol_w);
                    if (!kGlu || j == 0)
                        tma_load_2d(dst + 2 * kPanel + j * kRows, &tm_rows, rows_mn(kMode) ? r0 : d, rows_mn(kMode) ? d : r0, full,
                                    pol_x);
                }
            }
            __syncwarp();
            if (++s == kStages) s = 0, ph ^= 1;
        }
        for (int i = 0; i < min(kStages, s1 - s0); ++i) {   // the last copies land before the CTA ends
            if (--s < 0) s = kStages - 1, ph ^= 1;
            await_end(smem_u32(&ctrl->full[s]), ph ^ 1, p);
        }
    } else if (warp <= 2) {
        // one thread for each panel of a stage
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(128, BT) | idesc_major(cols_mn(kMode), rows_mn(kMode));
            const int j = warp - 1;
            const uint64_t a0 = operand_desc(base + j * kPanel);
            const uint64_t x0 = operand_desc(base + 2 * kPanel + (kGlu ? 0 : j) * kRows);
            int s = 0, b = 0;
            uint32_t ph = 0, tph = 1;
            for (int st = s0; st < s1; ++st) {
                if (!await(smem_u32(&ctrl->full[s]), ph, abort_flag, p)) break;
                if (kGlu || 2 * st + j < DB) {
                    if (!await(smem_u32(&ctrl->tempty[j][b]), tph, abort_flag, p)) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_e4m3(tmem + (j * kBufs + b) * BT, a0 + s * (kStage / 16) + kk * operand_step<cols_mn(kMode)>(),
                                  x0 + s * (kStage / 16) + kk * operand_step<rows_mn(kMode)>(), idesc, kk > 0);
                    umma_commit(smem_u32(&ctrl->tfull[j][b]));
                }
                umma_commit(smem_u32(&ctrl->empty[s]));
                if (++s == kStages) s = 0, ph ^= 1;
                if (++b == kBufs) b = 0, tph ^= 1;
            }
            if (s1 > s0) await_end(smem_u32(&ctrl->empty[s ? s - 1 : kStages - 1]), s ? ph : ph ^ 1, p);
        }
    } else if (warp == 3) {
        // the product of both scales for each row of each panel (weight's: the row's, and the column's apart)
        for (int st = s0, ch = 0; st < s1; st += kChunk / 2, ++ch) {
            const int slot = ch & 1;
            if (!await(smem_u32(&ctrl->sempty[slot]), ((ch >> 1) & 1) ^ 1, abort_flag, p)) break;
            float *sc = ctrl->sc[slot];
            if (kMode == kWeight) {
                const int r = r0 + 4 * (int)lane, c = tc * 128 + 4 * (int)lane, n = min(kChunk, DB - 2 * st);
                for (int j = 0; j < n; ++j) {
                    const int64_t b = 2 * st + j;
                    copy_scales(sc + j * (BT + 4) + 4 * lane, p.row_sf + b * p.rs_blk + r, r < p.R);
                    copy_scales(&ctrl->lane_sc[slot][j * 128 + 4 * lane], p.col_sf + b * p.cs_blk + c, c < p.C);
                }
                arrive_when_copied(smem_u32(&ctrl->sfull[slot]));
                continue;
            }
            constexpr int kBlocks = kGlu ? kChunk / 2 : kChunk, kEach = 32 / kBlocks;   // blocks of a chunk, rows of a load
            const int j = lane % kBlocks, b = (kGlu ? st : 2 * st) + j, sub = lane / kBlocks;
            float g = 0.0f, u = 0.0f;
            if (b < DB) {
                g = p.col_sf[tc * p.cs_col + b * p.cs_blk];
                if (kGlu) u = p.col_sf[(tc + p.C / 128) * p.cs_col + b * p.cs_blk];
            }
            float v[BT / kEach];
#pragma unroll
            for (int i = 0; i < BT / kEach; ++i) {
                const int r = r0 + sub + kEach * i;
                v[i] = b < DB && r < p.R ? p.row_sf[(int64_t)r * p.rs_row + b] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < BT / kEach; ++i) {
                sc[(kGlu ? 2 * j : j) * (BT + 4) + sub + kEach * i] = v[i] * g;
                if (kGlu) sc[(2 * j + 1) * (BT + 4) + sub + kEach * i] = v[i] * u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctrl->sfull[slot]));
        }
    } else {
        const int set = (warp - kSmallFold0) >> 2, q = warp & 3;
        const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + set * kBufs * BT;
        constexpr int kStep = BT < 32 ? BT : 32;
        float acc[BT];
#pragma unroll
        for (int i = 0; i < BT; ++i) acc[i] = 0.0f;
        for (int it = 0, st = s0; st < s1; ++st, ++it) {
            const int slot = (it >> 2) & 1, b = it % kBufs;
            if ((it & 3) == 0 && !await(smem_u32(&ctrl->sfull[slot]), (it >> 3) & 1, abort_flag, p)) break;
            if (kGlu || 2 * st + set < DB) {
                const int j = 2 * (it & 3) + set;
                const uint32_t sc = smem_u32(ctrl->sc[slot] + j * (BT + 4));
                const float mine = kMode == kWeight ? ctrl->lane_sc[slot][j * 128 + q * 32 + lane] : 1.0f;
                if (!await(smem_u32(&ctrl->tfull[set][b]), (it / kBufs) & 1, abort_flag, p)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < BT; c += kStep) {
                    float v[kStep];
                    if constexpr (kStep == 32) tmem_ld32(t + b * BT + c, v);
                    else tmem_ld16(t + b * BT + c, v);
                    tmem_ld_wait();
                    if (c + kStep == BT) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&ctrl->tempty[set][b]));
                    }
#pragma unroll
                    for (int i = 0; i < kStep; i += 4) {
                        const uint4 k = ld_shared16(sc + 4 * (c + i));
                        float4 f = make_float4(__uint_as_float(k.x), __uint_as_float(k.y), __uint_as_float(k.z), __uint_as_float(k.w));
                        if (kMode == kWeight) f.x *= mine, f.y *= mine, f.z *= mine, f.w *= mine;
                        acc[c + i] = fmaf(v[i], f.x, acc[c + i]);
                        acc[c + i + 1] = fmaf(v[i + 1], f.y, acc[c + i + 1]);
                        acc[c + i + 2] = fmaf(v[i + 2], f.z, acc[c + i + 2]);
                        acc[c + i + 3] = fmaf(v[i + 3], f.w, acc[c + i + 3]);
                    }
                }
            }
            if ((it & 3) == 3) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctrl->sempty[slot]));
            }
        }
        if (kSend) {
            // row i's sums to the CTA that joins it: i % split, where it is row i / split
            __syncwarp();
            cluster_wait();
            const uint32_t bar = smem_u32(&ctrl->sums), per = (rows + split - 1) / split;
            const uint32_t to = smem_u32(sent) + (rank * per * 256 + set * 128 + q * 32 + lane) * 4;
#pragma unroll
            for (int i = 0; i < BT; ++i)
                if (i < rows) {
                    const uint32_t who = i & (split - 1);
                    send(mapa_shared(to + (i / split) * 1024, who), acc[i], mapa_shared(bar, who));
                }
            cluster_arrive();
        } else {
            // every MMA of the CTA is done (both sets have seen theirs): the stages' memory takes the sums [set][row][128]
            asm volatile("bar.sync 1, 256;" ::: "memory");
            float *part = reinterpret_cast<float *>(smem_raw + (base - raw)) + (size_t)set * BT * 128 + q * 32 + lane;
#pragma unroll
            for (int i = 0; i < BT; ++i)
                if (i < rows) part[i * 128] = acc[i];
            if (!kSplit) asm volatile("bar.sync 1, 256;" ::: "memory");
        }
    }
    __syncwarp();
    if (kSend) {
        if (warp < kSmallFold0) cluster_wait(), cluster_arrive();
    } else if (kSplit) {
        cluster_sync();
    }
    // join the sums, in rank order: a warp takes rows of the tile, a lane four columns
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (warp >= kSmallFold0 && kSend) {
        if ((int)rank < rows && await(smem_u32(&ctrl->sums), 0, abort_flag, p)) {
            for (int k = warp - kSmallFold0; k * split + (int)rank < rows; k += 8) {
                const int64_t row = (int64_t)r0 + k * split + rank;
                float4 a = none, u = none, add = none;
                if (p.add && tc * 128 + 4 * (int)lane < p.C) add = load4(p, row, tc * 128 + 4 * (int)lane);
                for (int r = 0; r < split; ++r) {
                    const float *from = sent + (r * ((rows + split - 1) / split) + k) * 256 + 4 * lane;
                    a = plus(a, *reinterpret_cast<const float4 *>(from));
                    u = plus(u, *reinterpret_cast<const float4 *>(from + 128));
                }
                finish4<kGlu>(p, a, u, add, row, tc);
            }
        }
    } else if (warp >= kSmallFold0) {
        constexpr int kTogether = BT >= 64 ? 4 : 1;   // rows on their way together
        const int step = 8 * split;
        for (int i0 = (warp - kSmallFold0) * split + (int)rank; i0 < rows; i0 += kTogether * step) {
            float4 sum[kTogether][2], add[kTogether];
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                sum[k][0] = sum[k][1] = add[k] = none;
                if (p.add && tc * 128 + 4 * (int)lane < p.C && i0 + k * step < rows) add[k] = load4(p, (int64_t)r0 + i0 + k * step, tc * 128 + 4 * (int)lane);
            }
            for (int r = 0; r < split; ++r) {
                float4 v[kTogether][2];
#pragma unroll
                for (int k = 0; k < kTogether; ++k) {
                    const uint32_t at = base + (uint32_t)((min(i0 + k * step, BT - 1) * 128 + 4 * lane) * 4);   // a row past the last is not stored
                    const uint32_t from = kSplit ? mapa_shared(at, r) : at;
                    v[k][0] = ld_cluster16(from);
                    v[k][1] = ld_cluster16(from + BT * 512);
                }
#pragma unroll
                for (int k = 0; k < kTogether; ++k) sum[k][0] = plus(sum[k][0], v[k][0]), sum[k][1] = plus(sum[k][1], v[k][1]);
            }
#pragma unroll
            for (int k = 0; k < kTogether; ++k)
                if (i0 + k * step < rows) finish4<kGlu>(p, sum[k][0], sum[k][1], add[k], (int64_t)r0 + i0 + k * step, tc);
        }
    }
    // where a wait gave up too, the sums on their way to this CTA land before it ends: every CTA sends them, and a barrier of the
    // cluster orders their start alone
    if (kSend && threadIdx.x == 0) await_end(smem_u32(&ctrl->sums), 0, p);
    __syncwarp();
    tc_fence_before();
    // no CTA leaves while another sends to it or reads from it
    if (kSend) {
        cluster_wait();
        __syncthreads();
    } else if (kSplit) {
        cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// ---- host ------------------------------------------------------------------
constexpr int kMaxFeatures = 1 << 20;

thread_local int armed_us = 0;   // a test's wait limit for this thread's next launch

int up_to(int64_t n, int m) { return (int)((n + m - 1) / m); }

bool valid(const moe_fp8_linear_config *c) {
    if (!c || c->in_features < 16 || c->in_features % 16 || c->in_features > kMaxFeatures) return false;
    if (c->out_features < 16 || c->out_features % 16 || c->out_features > kMaxFeatures) return false;
    if (c->act != MOE_ACT_NONE && c->act != MOE_ACT_SWIGLU) return false;
    if (c->act == MOE_ACT_SWIGLU && c->out_features % 256) return false;
    if (c->quant != MOE_QUANT_NONE && (c->quant != MOE_QUANT_FP8_128 || c->act != MOE_ACT_SWIGLU)) return false;
    return valid_dtype(c->out_dtype) && c->act_clamp > 0.0f;
}

// Rows of a 16-byte aligned matrix, with a pitch that keeps them so.
bool rows_ok(const void *p, int64_t ld, int64_t cols, size_t es) {
    return p && aligned_to(p, 16) && ld >= cols && ld * (int64_t)es % 16 == 0;
}
// Whether two matrices of `rows` x `cols` elements share an element or may: apart in memory, or columns of the same rows that do not
// meet, they do not.
bool overlap(const void *p, int64_t ld_p, const void *q, int64_t ld_q, int64_t rows, int64_t cols, size_t es) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q), row = (uintptr_t)cols * es;
    const uintptr_t pitch_a = (uintptr_t)ld_p * es, pitch_b = (uintptr_t)ld_q * es, last = (uintptr_t)rows - 1;
    if (a + last * pitch_a + row <= b || b + last * pitch_b + row <= a) return false;
    if (rows == 1 || pitch_a != pitch_b) return true;
    const uintptr_t off = a < b ? (b - a) % pitch_a : (a - b) % pitch_a;   // from a row of the one to the next of the other
    return off < row || pitch_a - off < row;
}
// An added matrix: absent, the output itself, row by row, or apart from it (tiles are read and stored in no fixed order).
bool add_ok(const void *add, int64_t ld, const void *out, int64_t ld_out, int64_t rows, int64_t cols, size_t es) {
    if (!add) return true;
    if (!rows_ok(add, ld, cols, es)) return false;
    return add == out ? ld == ld_out || rows == 1 : !overlap(add, ld, out, ld_out, rows, cols, es);
}

template <int kMode>
cudaError_t launch_wide(const CUtensorMap &rows, const CUtensorMap &cols, const CUtensorMap &add, const CUtensorMap &out, const Fp8Params &p, int dev, cudaStream_t s) {
    static std::atomic<int> resident[32];   // CTA pairs that the device holds at once
    static std::atomic<uint32_t> smem_set{0};
    cudaError_t e = smem_limit_once(reinterpret_cast<const void *>(fp8_wide_kernel<kMode>), wide_smem<kMode>(), smem_set);
    if (e != cudaSuccess) return e;
    int pairs = resident[dev].load(std::memory_order_acquire);
    if (!pairs) {
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute a[1];
        a[0].id = cudaLaunchAttributeClusterDimension;
        a[0].val.clusterDim.x = 2, a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
        c.gridDim = dim3(sm_count(dev) & ~1);
        c.blockDim = dim3(kWideThreads);
        c.dynamicSmemBytes = wide_smem<kMode>();
        c.attrs = a, c.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&pairs, fp8_wide_kernel<kMode>, &c);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorLaunchOutOfResources;
        resident[dev].store(pairs, std::memory_order_release);
    }
    const int64_t tiles = (int64_t)p.tiles_r * p.tiles_c;
    return launch(fp8_wide_kernel<kMode>, 2u * (unsigned)std::min<int64_t>(pairs, tiles), kWideThreads, wide_smem<kMode>(), 2, s,
                  rows, cols, add, out, p);
}

template <int kMode, int BT, bool kSplit>
cudaError_t launch_small(const CUtensorMap &rows, const CUtensorMap &cols, Fp8Params p, cudaStream_t s) {
    static std::atomic<uint32_t> smem_set{0};
    constexpr size_t kFixed = 1024 + sizeof(SmallCtrl<kMode, BT>), kStage = small_stage<kMode, BT>(), kRoom = BT == 16 ? kSmHalf : kSmAll;
    constexpr size_t kSent = small_sends<BT, kSplit>() ? sent_bytes(BT, 8) : 0;
    static_assert(kFixed + kSent + 2 * kStage <= kRoom, "shared memory");
    cudaError_t e = smem_limit_once(reinterpret_cast<const void *>(fp8_small_kernel<kMode, BT, kSplit>), kRoom, smem_set);
    if (e != cudaSuccess) return e;
    const size_t sent = kSent ? sent_bytes(std::min(p.R, BT), p.split) : 0;
    p.stages = (int)std::min<size_t>(kMaxStages, (kRoom - kFixed - sent) / kStage);
    return launch(fp8_small_kernel<kMode, BT, kSplit>, (unsigned)(p.tiles_r * p.tiles_c * p.split), kSmallThreads,
                  kFixed + p.stages * kStage + sent, p.split, s, rows, cols, p);
}
template <int kMode, int BT>
cudaError_t launch_small(const CUtensorMap &rows, const CUtensorMap &cols, const Fp8Params &p, cudaStream_t s) {
    return p.split > 1 ? launch_small<kMode, BT, true>(rows, cols, p, s) : launch_small<kMode, BT, false>(rows, cols, p, s);
}

// Clusters of `split` CTAs, one an SM, that the device holds at once.
int resident_clusters(int dev, int split) {
    static std::atomic<int> known[32][4];
    if (split == 1) return sm_count(dev);
    std::atomic<int> &slot = known[dev][split == 2 ? 1 : split == 4 ? 2 : 3];
    int n = slot.load(std::memory_order_acquire);
    if (!n) {
        static std::atomic<uint32_t> smem_set{0};
        const auto kernel = fp8_small_kernel<kForward, 64, true>;
        if (smem_limit_once(reinterpret_cast<const void *>(kernel), kSmAll, smem_set) != cudaSuccess) return 0;
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute a[1];
        a[0].id = cudaLaunchAttributeClusterDimension;
        a[0].val.clusterDim.x = split, a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
        c.gridDim = dim3(sm_count(dev) / split * split);
        c.blockDim = dim3(kSmallThreads);
        c.dynamicSmemBytes = kSmAll;
        c.attrs = a, c.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess || n < 1) return 0;
        slot.store(n, std::memory_order_release);
    }
    return n;
}

// Which kernel, and how: rows of a tile (0: the wide kernel) and CTAs to a tile, by what they are estimated to take, in ns, from
// what was measured: a panel of 128 x 128 weights with 32 rows 200, with 64 245 (each wave of CTAs 2000 more, joining a cluster's
// sums 1300 and 50 a row); of a weight's gradient 500; a block of a wide tile 430, of a weight's gradient 600 (each wave of
// CTA pairs 2500, the launch 1500).  Sides of it: 128 x 7168 x 2048 11.8 us wide, 8.5 in 64s; 129 rows 13.0 wide, 14.5 in 64s;
// 512 x 576 x 7168 25.7 wide, 16.4 in 64s, 14.2 with two CTAs to a tile; 999 x 2064 x 4176 25 us in 128s, 22 wide.
struct Plan {
    int bt, split;
};
Plan plan_for(int mode, int64_t R, int64_t C, int DB, int sms, int dev) {
    const int64_t panels = mode == kSwiglu ? 2 * (int64_t)DB : DB, stages = (panels + 1) / 2, cols = up_to(C, 128);
    // two CTAs an SM (one, with more stages or registers, 13 to 15 us for one token's 4096 x 7168, two 8.6); as many to a tile as
    // fill the SMs once, the next call's beside them
    if (mode != kWeight && R <= 16) {
        int split = 1;
        while (split < 8 && cols * split * 2 <= sms && stages >= 4 * split) split *= 2;
        return {16, split};
    }
    const int64_t pairs = sms / 2, tiles = up_to(R, 256) * (int64_t)up_to(C, mode == kSwiglu ? 128 : 256);
    int64_t best = (tiles + pairs - 1) / pairs * ((int64_t)DB * (mode == kWeight ? 600 : 430) + 2500) + 1500;
    Plan plan{0, 1};
    for (int bt = mode == kWeight ? 128 : 32; bt <= (mode == kWeight ? 128 : 64); bt *= 2) {
        const int64_t each = mode == kWeight ? 500 : bt == 32 ? 200 : 245, n = up_to(R, bt) * cols;
        for (int split = 1; split <= (mode == kWeight ? 4 : 8); split *= 2) {
            if (split > 1 && stages < 2 * split) break;
            const int64_t room = resident_clusters(dev, split);
            if (!room || (split > 1 && n > room)) break;
            const int64_t cost = (n + room - 1) / room * ((panels + split - 1) / split * each + 2000) +
                                 (split > 1 ? 1300 + 50 * std::min<int64_t>(R, bt) : 0);
            if (cost < best) best = cost, plan = {bt, split};
        }
    }
    return plan;
}

// rows [R x D] and cols [C' x D] codes; ld: pitch of the matrix as stored.
template <int kMode>
int run(const uint8_t *rows, int64_t ld_rows, const uint8_t *cols, int64_t ld_cols, int64_t D, Fp8Params p, cudaStream_t s) {
    const int dev = this_device();
    const int sms = dev < 0 ? 0 : sm_count(dev);
    if (!sms) return MOE_ERR_CUDA;
    p.DB = up_to(D, 128);
    p.wait_us = armed_us, armed_us = 0;
    const int wt = kMode == kSwiglu ? 2 * p.C : p.C;   // rows of W
    const Plan plan = plan_for(kMode, p.R, p.C, p.DB, sms, dev);
    const uint32_t box = plan.bt ? plan.bt : 128;
    CUtensorMap mr, mc;
    if (!(rows_mn(kMode) ? encode_map(&mr, rows, p.R, D, ld_rows, 128, 128) : encode_map(&mr, rows, D, p.R, ld_rows, 128, box)) ||
        !(cols_mn(kMode) ? encode_map(&mc, cols, wt, D, ld_cols, 128, 128) : encode_map(&mc, cols, D, wt, ld_cols, 128, 128)))
        return MOE_ERR_CUDA;
    cudaError_t e;
    if (!plan.bt) {
        p.tiles_r = up_to(p.R, 256);
        p.tiles_c = up_to(p.C, kMode == kSwiglu ? 128 : 256);
        const int es = p.f32 ? 4 : 2;
        p.out_stages = p.sf ? 0 : kMode != kSwiglu && p.f32 ? 2 : 1;
        CUtensorMap mo = mr, ma = mr;
        if (p.out_stages && (!encode_map(&mo, p.out, (uint64_t)p.C * es, p.R, p.ld_out * es, 128, 128) ||
                             (p.add && !encode_map(&ma, p.add, (uint64_t)p.C * es, p.R, p.ld_add * es, 128, 128))))
            return MOE_ERR_CUDA;
        e = launch_wide<kMode>(mr, mc, ma, mo, p, dev, s);
    } else {
        p.tiles_r = up_to(p.R, plan.bt);
        p.tiles_c = up_to(p.C, 128);
        p.split = plan.split;
        if constexpr (kMode == kWeight)
            e = launch_small<kMode, 128>(mr, mc, p, s);
        else
            e = plan.bt == 16   ? launch_small<kMode, 16>(mr, mc, p, s)
                : plan.bt == 32 ? launch_small<kMode, 32>(mr, mc, p, s)
                                : launch_small<kMode, 64>(mr, mc, p, s);
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_fp8_linear_forward(const moe_fp8_linear_config *cfg, int num_tokens, const void *x, int64_t ld_x, const float *x_sf,
                           const void *w, const float *w_sf, const void *add, int64_t ld_add, void *y, int64_t ld_y, float *y_sf,
                           void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const bool glu = cfg->act == MOE_ACT_SWIGLU, quant = cfg->quant != MOE_QUANT_NONE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_tokens == 0) return MOE_OK;
    if (quant ? !y_sf || add : y_sf != nullptr) return MOE_ERR_INVALID_ARG;
    const int64_t K = cfg->in_features, N = cfg->out_features, n = glu ? N / 2 : N;
    const size_t es = quant ? 1 : dtype_bytes(cfg->out_dtype);
    if (!rows_ok(x, ld_x, K, 1) || !rows_ok(w, K, K, 1) || !rows_ok(y, ld_y, n, es) || !add_ok(add, ld_add, y, ld_y, num_tokens, n, es))
        return MOE_ERR_INVALID_ARG;
    if (!x_sf || !w_sf || !aligned_to(x_sf, 4) || !aligned_to(w_sf, 4) || !aligned_to(y_sf, 4)) return MOE_ERR_INVALID_ARG;
    Fp8Params p{};
    p.row_sf = x_sf, p.col_sf = w_sf;
    p.rs_row = p.cs_col = up_to(K, 128);
    p.rs_blk = p.cs_blk = 1;
    p.add = add, p.ld_add = ld_add, p.out = y, p.ld_out = ld_y, p.sf = y_sf;
    p.R = num_tokens, p.C = (int)n, p.f32 = cfg->out_dtype == MOE_DTYPE_F32, p.clamp = cfg->act_clamp;
    const uint8_t *a = static_cast<const uint8_t *>(x), *b = static_cast<const uint8_t *>(w);
    return glu ? run<kSwiglu>(a, ld_x, b, K, K, p, s) : run<kForward>(a, ld_x, b, K, K, p, s);
}

int moe_fp8_linear_backward_input(const moe_fp8_linear_config *cfg, int num_tokens, const void *dy, int64_t ld_dy,
                                  const float *dy_sf, const void *w, const float *w_sf, const void *add, int64_t ld_add, void *dx,
                                  int64_t ld_dx, void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    const int64_t K = cfg->in_features, N = cfg->out_features;
    const size_t es = dtype_bytes(cfg->out_dtype);
    if (!rows_ok(dy, ld_dy, N, 1) || !rows_ok(w, K, K, 1) || !rows_ok(dx, ld_dx, K, es) || !add_ok(add, ld_add, dx, ld_dx, num_tokens, K, es))
        return MOE_ERR_INVALID_ARG;
    if (!dy_sf || !w_sf || !aligned_to(dy_sf, 4) || !aligned_to(w_sf, 4)) return MOE_ERR_INVALID_ARG;
    Fp8Params p{};
    p.row_sf = dy_sf, p.col_sf = w_sf;
    p.rs_row = up_to(N, 128), p.rs_blk = 1;
    p.cs_col = 1, p.cs_blk = up_to(K, 128);
    p.add = add, p.ld_add = ld_add, p.out = dx, p.ld_out = ld_dx;
    p.R = num_tokens, p.C = (int)K, p.f32 = cfg->out_dtype == MOE_DTYPE_F32;
    return run<kInput>(static_cast<const uint8_t *>(dy), ld_dy, static_cast<const uint8_t *>(w), K, N, p,
                       static_cast<cudaStream_t>(stream));
}

int moe_fp8_linear_backward_weight(const moe_fp8_linear_config *cfg, int num_tokens, const void *dy, int64_t ld_dy,
                                   const float *dy_sf, const void *x, int64_t ld_x, const float *x_sf, const float *add,
                                   int64_t ld_add, float *dw, int64_t ld_dw, void *stream) {
    if (!valid(cfg) || num_tokens < 0) return MOE_ERR_INVALID_ARG;
    const int64_t K = cfg->in_features, N = cfg->out_features;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!rows_ok(dw, ld_dw, K, 4) || !add_ok(add, ld_add, dw, ld_dw, N, K, 4)) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) {   // nothing is summed
        const cudaError_t e = !add       ? cudaMemset2DAsync(dw, ld_dw * 4, 0, K * 4, N, s)
                              : add != dw ? cudaMemcpy2DAsync(dw, ld_dw * 4, add, ld_add * 4, K * 4, N, cudaMemcpyDeviceToDevice, s)
                                          : cudaSuccess;
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    if (!rows_ok(dy, ld_dy, N, 1) || !rows_ok(x, ld_x, K, 1)) return MOE_ERR_INVALID_ARG;
    if (!dy_sf || !x_sf || !aligned_to(dy_sf, 16) || !aligned_to(x_sf, 16)) return MOE_ERR_INVALID_ARG;
    Fp8Params p{};
    p.row_sf = dy_sf, p.col_sf = x_sf;
    p.rs_row = p.cs_col = 1;
    p.rs_blk = N, p.cs_blk = K;
    p.add = add, p.ld_add = ld_add, p.out = dw, p.ld_out = ld_dw;
    p.R = (int)N, p.C = (int)K, p.f32 = 1;
    return run<kWeight>(static_cast<const uint8_t *>(dy), ld_dy, static_cast<const uint8_t *>(x), ld_x, num_tokens, p, s);
}

int moe_fp8_linear_test_arm_timeout(int wait_limit_us) {
    if (wait_limit_us < 1) return MOE_ERR_INVALID_ARG;
    armed_us = wait_limit_us;
    return MOE_OK;
}

int moe_fp8_linear_status(void) {
    int w[kErrWords] = {};
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpyFromSymbol(w, g_status, sizeof w) != cudaSuccess) return MOE_ERR_CUDA;
    if (!w[0]) return MOE_OK;
    const int zero[kErrWords] = {};
    if (cudaMemcpyToSymbol(g_status, zero, sizeof zero) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
