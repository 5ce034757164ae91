// moe_norm.cu -- the norms after one block and before the next, fused with the
// gate, the residual sum and the expert layer's input quantisation, forward
// and backward (formulas in include/moe.h).
//
// Both directions are bound by reading and writing the [T, H] tensors once.  A
// row lives in the registers of the threads that own its columns, 8 columns
// (one chunk) to a thread at a time, from the first load to the last store, so
// every input is read once and every output written once whatever the norms in
// between need.  Sums over a row are f32: 8 terms a chunk in order, then the
// warp's tree, then the warps'.
//
// Forward: a row's time is two reductions one after the other, each a barrier,
// so what counts is that memory is busy meanwhile: the next rows come through
// private slots of shared memory by asynchronous copies, and two CTAs share an
// SM.  4096 rows of 7168 bf16 with codes and normed output: 44.2 us, 6.0 TB/s
// (a simple kernel with a CTA a row 135); 1023 rows of 4096 to UE8M0 codes
// 10.5 us; one row 3.9 us, which is the latency of a launch, three dependent
// trips to memory and shared memory and two barriers.
//
// Backward: four tensors come in and two go out, with one reduction after two
// of them have arrived and one after the fourth; the column sums stay in
// registers (two per column are enough: the gradients of w_post and of a
// channel's gate are the same sum times the other one) and are joined by a
// second kernel in a fixed order.  4096 rows of 7168 bf16: 76.0 us, 4.6 TB/s,
// 66 of them in the main kernel (a simple kernel 719); 1777 rows of 1001 f32
// by element: 13.9 us.
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

// How a thread's 8 * NV columns lie in the row.
//   kVec: chunks of 8 columns, 16-byte accesses (every row and parameter 16-byte aligned, H % 8 == 0);
//   kChunk: the same chunks by element (any alignment; the quantised outputs need chunks);
//   kStride: columns tid, tid + threads, ... by element: what an odd width or pitch gets, coalesced.
enum Map { kVec, kChunk, kStride };

template <Map M>
__device__ __forceinline__ int column(int i, int j, int tr, int threads) {
    return M == kStride ? (i * 8 + j) * threads + tr : (i * threads + tr) * 8 + j;
}

// 8 columns of a row as f32 (zero past the row's end).
template <Map M, class S>
__device__ __forceinline__ void load8(F8 &v, const S *row, int i, int tr, int threads, int H) {
    if (M == kVec) {
        const int c = column<M>(i, 0, tr, threads);
        if (c < H) {
            Raw8<S> r;
            r.load(row + c);
            r.get(v);
        } else {
            v.fill(0.0f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<M>(i, j, tr, threads);
            v.put(j, c < H ? to_f32(row[c]) : 0.0f);
        }
    }
}

template <Map M, class S>
__device__ __forceinline__ void store8(S *row, const F8 &v, int i, int tr, int threads, int H) {
    if (M == kStride) {
        S *at = row + column<M>(i, 0, tr, threads);
#pragma unroll
        for (int j = 0; j < 8; ++j, at += threads)
            if (column<M>(i, j, tr, threads) < H) *at = from_f32<S>(v.get(j));
    } else if (M == kVec) {
        const int c = column<M>(i, 0, tr, threads);
        if (c < H) {
            Raw8<S> r;
            r.set(v);
            r.store(row + c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<M>(i, j, tr, threads);
            if (c < H) row[c] = from_f32<S>(v.get(j));
        }
    }
}

// The same for parameters, whose type is known at run time only (uniform branch).
template <Map M>
__device__ __forceinline__ void load_param8(F8 &v, const void *w, bool f32, int i, int tr, int threads, int H) {
    if (f32) load8<M>(v, static_cast<const float *>(w), i, tr, threads, H);
    else load8<M>(v, static_cast<const bf16 *>(w), i, tr, threads, H);
}
__device__ __forceinline__ float load_param(const void *w, bool f32, int64_t i) {
    return f32 ? static_cast<const float *>(w)[i] : to_f32(static_cast<const bf16 *>(w)[i]);
}

// Sum over a row's threads in a fixed order: a warp, or the CTA (`red` one float per warp, not in use).
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if (kWarpRow) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f);
}

// The same for R rows of the CTA behind one barrier (`red` R floats per warp).
template <int R>
__device__ __forceinline__ void row_sums(float (&v)[R], float *red) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_sum(v[r]);
    if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) red[r * 32 + (threadIdx.x >> 5)] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_sum(lane < (int)(blockDim.x >> 5) ? red[r * 32 + lane] : 0.0f);
}

struct NormFwd {
    moe_norm_io io;
    int T, H, quant, gate, slots;
    bool param_f32;
    float eps, residual_scale;
};

// A thread's part of one stream tensor's row, on its way while earlier rows are worked on.  With aligned rows (kRing) it
// comes through shared memory by asynchronous 16-byte copies, into slots that no other thread touches: the waits are the
// thread's own, and a slot can be refilled as soon as the thread has read it.  Else it is loaded into registers: by
// element one to an element, because packing two at once would wait for them there and then (4096 x 5001 bf16 forward:
// 270 us against 79).
template <class S, int NV, Map M, bool kRing>
struct Feed {
    Raw8<S> v[kRing || M != kVec ? 1 : NV];
    S e[M != kVec ? NV * 8 : 1];
    uint32_t slots;   // kRing: shared address of [slot][NV][threads] 16 (bf16) or 32 (f32) bytes
    __device__ __forceinline__ uint32_t at(int slot, int i, int tr, int threads) const {
        return slots + ((slot * NV + i) * threads + tr) * (uint32_t)(8 * sizeof(S));
    }
    __device__ __forceinline__ void fetch(const void *base, int64_t ld, int64_t t, int slot, int tr, int threads, int H) {
        if (!base) return;
        const S *row = static_cast<const S *>(base) + t * ld;
        const S *at_c = row + column<M>(0, 0, tr, threads);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (M == kVec) {
                const int c = column<M>(i, 0, tr, threads);
                if (kRing) {
                    if (c < H) copy_async<8 * sizeof(S)>(at(slot, i, tr, threads), row + c);
                } else if (c < H) {
                    v[kRing || M != kVec ? 0 : i].load_once(row + c);
                } else {
                    v[kRing || M != kVec ? 0 : i].zero();
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = column<M>(i, j, tr, threads);
                    if (M == kStride) {
                        e[M != kVec ? i * 8 + j : 0] = c < H ? *at_c : from_f32<S>(0.0f);
                        at_c += threads;
                    } else {
                        e[M != kVec ? i * 8 + j : 0] = c < H ? row[c] : from_f32<S>(0.0f);
                    }
                }
            }
        }
    }
    // Zeros where no copy will write: the chunks past the row's end, and rows past the last one.
    __device__ __forceinline__ void clear(int n, int tr, int threads, int H) {
        if (kRing) {
            for (int slot = 0; slot < n; ++slot)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    for (int b = 0; b < (int)sizeof(S) / 2; ++b)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at(slot, i, tr, threads) + 16 * b), "r"(0)
                                     : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (M == kVec) v[kRing || M != kVec ? 0 : i].zero();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (M != kVec) e[M != kVec ? i * 8 + j : 0] = from_f32<S>(0.0f);
            }
        }
    }
    __device__ __forceinline__ void get(F8 &f, int i, int slot, int tr, int threads) const {
        if (kRing) {
            Raw8<S> r;
            r.load_shared(at(slot, i, tr, threads));
            r.get(f);
        } else if (M == kVec) {
            v[kRing || M != kVec ? 0 : i].get(f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f.put(j, to_f32(e[M != kVec ? i * 8 + j : 0]));
        }
    }
};
// Where a CTA that walks rows keeps its columns' parameters: in registers, in shared memory (each thread its own), or
// nowhere (loaded for every row).
enum Keep { kNone, kRegs, kShared };
template <int NV, Keep K>
struct Params {
    F8 reg[K == kRegs ? NV : 1];
    uint32_t base;   // kShared: shared address of [NV][2][threads] 16 bytes
    static constexpr int kBytes = K == kShared ? NV * 32 : 0;   // a thread's
    __device__ __forceinline__ uint32_t at(int i, int half, int tr, int threads) const {
        return base + ((i * 2 + half) * threads + tr) * 16;
    }
    __device__ __forceinline__ void set(int i, const F8 &v, int tr, int threads) {
        if (K == kRegs) reg[K == kRegs ? i : 0] = v;
        if (K == kShared)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at(i, h, tr, threads)), "f"(v.p[2 * h].x),
                             "f"(v.p[2 * h].y), "f"(v.p[2 * h + 1].x), "f"(v.p[2 * h + 1].y)
                             : "memory");
    }
    __device__ __forceinline__ void get(F8 &v, int i, int tr, int threads) const {
        if (K == kRegs) v = reg[K == kRegs ? i : 0];
        if (K == kShared)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 q = ld_shared16(at(i, h, tr, threads));
                v.p[2 * h] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
                v.p[2 * h + 1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
            }
    }
};

constexpr int kMaxSlots = 4;
// Waits until at most n of this thread's groups of copies are under way.
__device__ __forceinline__ void wait_groups(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;   // 2 kMaxSlots - 1
    }
}
__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Codes and scale of a thread's chunk at column c.  A group is 16 (of 128 columns) or 4 (of 32) neighbouring chunks,
// all of them in the row or none; every lane of the warp calls.
__device__ __forceinline__ void quantise8(const NormFwd &p, F8 v, int64_t t, int c, int tr) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v.get(j)));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    float inv;
    if (p.quant == MOE_QUANT_FP8_128) {
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
        const Fp8Scale sc = fp8_scale(amax, v);
        inv = sc.inv;
        if (c < p.H && (tr & 15) == 0) static_cast<float *>(p.io.sf)[t * (p.H / 128) + c / 128] = sc.sf;
    } else {
        const int code = ue8m0_code(amax);
        inv = ue8m0_inverse(code);
        if (c < p.H && (tr & 3) == 0) static_cast<uint8_t *>(p.io.sf)[t * (p.H / 32) + c / 32] = (uint8_t)code;
    }
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 s = __fmul2_rn(v.p[j], pair(inv));
        q[j] = e4m3x2(s.x, s.y);
    }
    if (c < p.H) *reinterpret_cast<uint2 *>(p.io.codes + t * p.H + c) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// A warp takes one row (kWarpRow), or a CTA rows b, b + CTAs, ... with the next `slots` rows on their way and (kKeep) its
// columns' parameters in registers.
template <class S, int NV, Map M, bool kWarpRow, Keep kKeep, int kMaxThreads, int kMinCtas>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas) norm_fwd_kernel(const __grid_constant__ NormFwd p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][2][32];
    constexpr bool kRing = M == kVec && !kWarpRow;
    launch_next();
    wait_for_previous();
    const int tr = kWarpRow ? threadIdx.x & 31 : threadIdx.x, threads = kWarpRow ? 32 : blockDim.x;
    const int H = p.H, slots = kRing ? p.slots : 1;
    const float inv_h = 1.0f / (float)H;
    int64_t t = kWarpRow ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    Feed<S, NV, M, kRing> res, y;
    res.slots = smem_u32(ring);
    y.slots = res.slots + (uint32_t)(slots * NV * threads * 8 * sizeof(S));
    if (kRing && H < NV * 8 * threads) {
        res.clear(slots, tr, threads, H);
        y.clear(slots, tr, threads, H);
    }
    auto fetch = [&](int64_t t, int slot) {
        if (t < p.T) {
            y.fetch(p.io.y, p.io.ld_y, t, slot, tr, threads, H);
            res.fetch(p.io.residual, p.io.ld_residual, t, slot, tr, threads, H);
        }
        if (kRing) commit_group();
    };
    // By element over 8192 columns no registers are left for a row ahead (4096 x 9001 bf16: 398 us, ahead and spilled 413).
    constexpr bool kAhead = !(M != kVec && !kWarpRow && kKeep == kNone);
    if (kAhead)
        for (int i = 0; i < slots; ++i) fetch(t + (int64_t)i * gridDim.x, i);
    // w_post times a channel's gate (1 where absent)
    auto load_post = [&](F8 &w, int i) {
        if (p.io.w_post) load_param8<M>(w, p.io.w_post, p.param_f32, i, tr, threads, H);
        else w.fill(1.0f);
        if (p.gate == MOE_GATE_CHANNEL) {
            F8 g;
            load_param8<M>(g, p.io.gate, p.param_f32, i, tr, threads, H);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.p[j] = __fmul2_rn(w.p[j], g.p[j]);
        }
    };
    Params<NV, kKeep> k_post, k_pre;
    k_post.base = res.slots + (uint32_t)(2 * slots * NV * threads * 8 * sizeof(S));
    k_pre.base = k_post.base + k_post.kBytes * threads;
    if (kKeep != kNone) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F8 w;
            if (p.io.y) {
                load_post(w, i);
                k_post.set(i, w, tr, threads);
            }
            if (p.io.w_pre) {
                load_param8<M>(w, p.io.w_pre, p.param_f32, i, tr, threads, H);
                k_pre.set(i, w, tr, threads);
            }
        }
    }
    auto token_gate = [&](int64_t t) {
        return p.gate == MOE_GATE_TOKEN && t < p.T ? load_param(p.io.gate, p.param_f32, t) : 1.0f;
    };
    float gate_ahead = token_gate(t);   // asked for one row ahead
    int turn = 0, slot = 0;   // the reductions of consecutive rows use different words: one barrier each is enough
    for (; t < p.T; t += gridDim.x, turn ^= 1, slot = slot + 1 == slots ? 0 : slot + 1) {
        const float gate = gate_ahead;
        if (!kWarpRow) gate_ahead = token_gate(t + gridDim.x);
        if (kRing) wait_groups(slots - 1);
        if (!kAhead) fetch(t, 0);
        F8 z[NV], u[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            res.get(z[i], i, slot, tr, threads);
            if (p.io.y) y.get(u[i], i, slot, tr, threads);
        }
        if (!kWarpRow && kAhead) fetch(t + (int64_t)slots * gridDim.x, slot);
        if (p.io.y) {
            float r1 = 1.0f;
            if (p.io.w_post) {
                float2 s1 = pair(0.0f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s1 = __ffma2_rn(u[i].p[j], u[i].p[j], s1);
                r1 = rsqrtf(fmaf(row_sum<kWarpRow>(s1.x + s1.y, red[0][turn]), inv_h, p.eps));
                if (tr == 0 && p.io.rstd_post) p.io.rstd_post[t] = r1;
            }
            r1 *= gate;
            S *h = static_cast<S *>(p.io.h) + t * p.io.ld_h;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F8 w;
                if (kKeep == kNone) load_post(w, i);
                else k_post.get(w, i, tr, threads);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    z[i].p[j] = __ffma2_rn(__fmul2_rn(u[i].p[j], w.p[j]), pair(r1),
                                           __fmul2_rn(pair(p.residual_scale), z[i].p[j]));
                store8<M>(h, z[i], i, tr, threads, H);
            }
        }
        if (p.io.w_pre) {
            float2 s2 = pair(0.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(z[i].p[j], z[i].p[j], s2);
            const float r2 = rsqrtf(fmaf(row_sum<kWarpRow>(s2.x + s2.y, red[1][turn]), inv_h, p.eps));
            if (tr == 0 && p.io.rstd_pre) p.io.rstd_pre[t] = r2;
            S *n = p.io.n ? static_cast<S *>(p.io.n) + t * p.io.ld_n : nullptr;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F8 w;
                if (kKeep == kNone) load_param8<M>(w, p.io.w_pre, p.param_f32, i, tr, threads, H);
                else k_pre.get(w, i, tr, threads);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i].p[j] = __fmul2_rn(__fmul2_rn(z[i].p[j], pair(r2)), w.p[j]);
                if (n) store8<M>(n, z[i], i, tr, threads, H);
                if (M != kStride && p.quant != MOE_QUANT_NONE) quantise8(p, z[i], t, column<M>(i, 0, tr, threads), tr);
            }
        }
        if (kWarpRow) break;
    }
}

// Where the backward pass keeps its parameters: in registers where a thread's rows and sums leave some.
constexpr Keep bwd_keep(int R, bool wide) {
    return wide ? kNone : R == 1 ? kRegs : kShared;
}
// Columns between the rows of partial sums.
__host__ __device__ __forceinline__ int64_t part_pitch(int H) { return (H + 31) / 32 * 32; }

struct NormBwd {
    moe_norm_grad_io io;
    float *part;   // [CTAs][2][part_pitch(H)]
    int T, H, gate, slots;
    bool param_f32;
    float residual_scale;
};

// With t = dn h, S2 = sum t w_pre, du = D yh and S1 = sum du gate w_post (a token's gate g left out of the sum):
//   D  = dh + r2 dn w_pre - h r2^3 S2 / H
//   dy = g r1 (D gate w_post - yh S1 / H)
// and only two sums over tokens are kept per column: P = sum r2 t is dw_pre, and A = sum g du gives dw_post (times a
// channel gate) and a channel's dgate (times w_post, g = 1) after the last row.
//
// CTA b takes rows b, b + CTAs, ...; every thread keeps its columns throughout, so the sums over tokens stay with it
// until the end: in registers, next to its columns' parameters, or for rows of over 8192 columns (kWide) in shared
// memory with everything else loaded where it is used.
template <class S, int NV, int R, Map M, bool kWide, int kMaxThreads, int kMinCtas>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas) norm_bwd_kernel(const __grid_constant__ NormBwd p) {
    extern __shared__ __align__(16) uint8_t ring[];
    float *wide_acc = reinterpret_cast<float *>(ring);   // kWide: [2][NV][8][threads]
    __shared__ float red[2][2][R * 32];
    const int tr = threadIdx.x, threads = blockDim.x, H = p.H;
    launch_next();
    wait_for_previous();
    const float inv_h = 1.0f / (float)H;
    const bool pre = p.io.dn != nullptr, block = p.io.y != nullptr, post = p.io.w_post != nullptr;
    const bool channel = p.gate == MOE_GATE_CHANNEL, token = p.gate == MOE_GATE_TOKEN;
    F8 acc[2][kWide ? 1 : NV];   // A, P
    // adds v * f to sum `which` of chunk i
    auto add = [&](int which, int i, int j, float2 v, float2 f) {   // pair j
        if (kWide) {
            float2 *at = reinterpret_cast<float2 *>(wide_acc) + ((which * NV + i) * 4 + j) * threads + tr;
            *at = __ffma2_rn(v, f, *at);
        } else {
            acc[which][kWide ? 0 : i].p[j] = __ffma2_rn(v, f, acc[which][kWide ? 0 : i].p[j]);
        }
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (kWide)
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float2 *>(wide_acc)[((k * NV + i) * 4 + j) * threads + tr] = pair(0.0f);
            else acc[k][kWide ? 0 : i].fill(0.0f);
        }
    // w_post times a channel's gate (1 where absent)
    auto load_scale = [&](F8 &w, int i) {
        if (post) load_param8<M>(w, p.io.w_post, p.param_f32, i, tr, threads, H);
        else w.fill(1.0f);
        if (channel) {
            F8 g;
            load_param8<M>(g, p.io.gate, p.param_f32, i, tr, threads, H);
#pragma unroll
            for (int j = 0; j < 4; ++j) w.p[j] = __fmul2_rn(w.p[j], g.p[j]);
        }
    };
    constexpr bool kRing = M == kVec && !kWide;
    const int slots = kRing ? p.slots : 1;
    Feed<S, NV, M, kRing> h[R], y[R], dh[R], dn[R];
    const uint32_t tensor = (uint32_t)(slots * NV * threads * 8 * sizeof(S));
#pragma unroll
    for (int r = 0; r < R; ++r) {
        h[r].slots = smem_u32(ring) + 4 * r * tensor;
        dn[r].slots = h[r].slots + tensor, dh[r].slots = dn[r].slots + tensor, y[r].slots = dh[r].slots + tensor;
        if (kRing && H == NV * 8 * threads) continue;   // every chunk is copied
        h[r].clear(slots, tr, threads, H), dn[r].clear(slots, tr, threads, H);
        dh[r].clear(slots, tr, threads, H), y[r].clear(slots, tr, threads, H);
    }
    // row r of the pass that begins at row t
    auto fetch_pre = [&](int64_t t, int slot, int r) {
        t += r * (int64_t)gridDim.x;
        if (t >= p.T || !pre) return;
        h[r].fetch(p.io.h, p.io.ld_h, t, slot, tr, threads, H);
        dn[r].fetch(p.io.dn, p.io.ld_dn, t, slot, tr, threads, H);
    };
    auto fetch_dh = [&](int64_t t, int slot, int r) {
        t += r * (int64_t)gridDim.x;
        if (t < p.T) dh[r].fetch(p.io.dh, p.io.ld_dh, t, slot, tr, threads, H);
    };
    auto fetch_y = [&](int64_t t, int slot, int r) {
        t += r * (int64_t)gridDim.x;
        if (t < p.T) y[r].fetch(p.io.y, p.io.ld_y, t, slot, tr, threads, H);
    };
    if (!kWide)
        for (int i = 0; i < slots; ++i) {
            const int64_t t = blockIdx.x + (int64_t)i * R * gridDim.x;
#pragma unroll
            for (int r = 0; r < R; ++r) fetch_pre(t, i, r), fetch_dh(t, i, r);
            if (kRing) commit_group();
#pragma unroll
            for (int r = 0; r < R; ++r) fetch_y(t, i, r);
            if (kRing) commit_group();
        }
    constexpr Keep kKeep = bwd_keep(R, kWide);
    Params<NV, kKeep> k_scale, k_pre;
    k_scale.base = smem_u32(ring) + (kRing ? 4 * R * tensor : 0);
    k_pre.base = k_scale.base + k_scale.kBytes * threads;
    if (kKeep != kNone) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F8 w;
            if (block) {
                load_scale(w, i);
                k_scale.set(i, w, tr, threads);
            }
            if (pre) {
                load_param8<M>(w, p.io.w_pre, p.param_f32, i, tr, threads, H);
                k_pre.set(i, w, tr, threads);
            }
        }
    }
    // the row's scalars, asked for one row ahead
    struct Scalars {
        float r1, r2, g;
    };
    auto scalars = [&](int64_t t) {
        Scalars s{1.0f, 0.0f, 1.0f};
        if (t < p.T) {
            if (post) s.r1 = p.io.rstd_post[t];
            if (pre) s.r2 = p.io.rstd_pre[t];
            if (token) s.g = load_param(p.io.gate, p.param_f32, t);
        }
        return s;
    };
    Scalars ahead[R];
#pragma unroll
    for (int r = 0; r < R; ++r) ahead[r] = scalars(blockIdx.x + r * (int64_t)gridDim.x);
    int slot = 0;
    int turn = 0;   // the reductions of consecutive passes use different words: one barrier each is enough
    const int64_t step = (int64_t)R * gridDim.x;
    for (int64_t t = blockIdx.x; t < p.T; t += step, turn ^= 1, slot = slot + 1 == slots ? 0 : slot + 1) {
        const int64_t next = kWide ? p.T : t + slots * step;
        const bool pair_of_rows = R == 2 && t + gridDim.x < p.T;   // the second row is there
        Scalars now[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            now[r] = ahead[r];
            ahead[r] = scalars(t + step + r * (int64_t)gridDim.x);
        }
        if (kRing) wait_groups(2 * slots - 1);   // all but y: a pass's copies are two groups
        F8 D[R][NV];   // of a second row that is not there: whatever it holds, nothing is summed or written
        if (pre) {
            float2 s2[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s2[r] = pair(0.0f);
                if (kWide) fetch_pre(t, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F8 w;
                if (kKeep != kNone) k_pre.get(w, i, tr, threads);
                else load_param8<M>(w, p.io.w_pre, p.param_f32, i, tr, threads, H);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r == 1 && !pair_of_rows) continue;
                    F8 hv, v;
                    dn[r].get(v, i, slot, tr, threads);
                    h[r].get(hv, i, slot, tr, threads);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 th = __fmul2_rn(v.p[j], hv.p[j]);
                        add(1, i, j, th, pair(now[r].r2));
                        s2[r] = __ffma2_rn(th, w.p[j], s2[r]);
                        D[r][i].p[j] = __fmul2_rn(__fmul2_rn(v.p[j], pair(now[r].r2)), w.p[j]);
                    }
                }
            }
            float back[R];
#pragma unroll
            for (int r = 0; r < R; ++r) back[r] = s2[r].x + s2[r].y;
            row_sums<R>(back, red[0][turn]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // r2^3 may leave the f32 range (rows beyond 2^42, rows of zeros under a tiny eps): h r2 and the rest do not
                back[r] = back[r] * -now[r].r2 * inv_h * now[r].r2;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    F8 hv;
                    h[r].get(hv, i, slot, tr, threads);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        D[r][i].p[j] = __ffma2_rn(__fmul2_rn(hv.p[j], pair(now[r].r2)), pair(back[r]), D[r][i].p[j]);
                }
                fetch_pre(next, slot, r);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < NV; ++i) D[r][i].fill(0.0f);
        }
        const float rs = block ? p.residual_scale : 1.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tt = t + r * (int64_t)gridDim.x;
            if (p.io.dh) {
                if (kWide) fetch_dh(t, 0, 0);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    F8 v;
                    dh[r].get(v, i, slot, tr, threads);
#pragma unroll
                    for (int j = 0; j < 4; ++j) D[r][i].p[j] = __fadd2_rn(D[r][i].p[j], v.p[j]);
                }
                fetch_dh(next, slot, r);
            }
            if (r == 1 && !pair_of_rows) continue;
            S *dres = static_cast<S *>(p.io.dresidual) + tt * p.io.ld_dresidual;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F8 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v.p[j] = __fmul2_rn(pair(rs), D[r][i].p[j]);
                store8<M>(dres, v, i, tr, threads, H);
            }
        }
        if (kRing) commit_group();
        if (!block) {
            if (kRing) commit_group();
            continue;
        }
        if (kRing) wait_groups(2 * slots - 1);   // y, which was asked for last
        float2 s1[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s1[r] = pair(0.0f);
            if (kWide) fetch_y(t, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F8 w;
            if (kKeep != kNone) k_scale.get(w, i, tr, threads);
            else load_scale(w, i);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r == 1 && !pair_of_rows) continue;
                F8 v;
                y[r].get(v, i, slot, tr, threads);
                const float gr = now[r].g * now[r].r1;   // r1 is applied to the sums
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 du = __fmul2_rn(D[r][i].p[j], v.p[j]);
                    add(0, i, j, du, pair(gr));
                    s1[r] = __ffma2_rn(du, w.p[j], s1[r]);
                    D[r][i].p[j] = __fmul2_rn(D[r][i].p[j], w.p[j]);
                }
            }
        }
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r] = s1[r].x + s1[r].y;
        if (post || token) row_sums<R>(sum, red[1][turn]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tt = t + r * (int64_t)gridDim.x;
            if (r == 0 || pair_of_rows) {
                const float s = sum[r] * now[r].r1, gr = now[r].g * now[r].r1;
                if (token && tr == 0) p.io.dgate[tt] = s;
                const float back = post ? -s * inv_h * now[r].r1 : 0.0f;
                S *dy = static_cast<S *>(p.io.dy) + tt * p.io.ld_dy;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    F8 v;
                    y[r].get(v, i, slot, tr, threads);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v.p[j] = __fmul2_rn(pair(gr), __ffma2_rn(v.p[j], pair(back), D[r][i].p[j]));
                    store8<M>(dy, v, i, tr, threads, H);
                }
            }
            fetch_y(next, slot, r);
        }
        if (kRing) commit_group();
    }
    const int64_t pitch = part_pitch(H);
    float *part = p.part + (int64_t)blockIdx.x * 2 * pitch;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? post || channel : pre)) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F8 v;
            if (kWide)
                for (int j = 0; j < 4; ++j)
                    v.p[j] = reinterpret_cast<float2 *>(wide_acc)[((k * NV + i) * 4 + j) * threads + tr];
            else v = acc[k][kWide ? 0 : i];
            store8<M>(part + k * pitch, v, i, tr, threads, H);
        }
    }
}

// Column sums of the partials, always in the same order: 32 columns a CTA, 8 lanes of 4 columns to a row; a thread takes
// every kRows-th row, then those are added in turn.  With 32 rows at a time the CTAs are small enough for the first ones
// to be in place beside the main kernel's.
template <int kRows>
__global__ void __launch_bounds__(kRows * 8) norm_bwd_sum_kernel(const __grid_constant__ NormBwd p, int parts) {
    __shared__ float sum[kRows][33];
    const int H = p.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.x & 1, col0 = (blockIdx.x >> 1) * 32;
    const bool channel = p.gate == MOE_GATE_CHANNEL;
    launch_next();
    wait_for_previous();
    if (which == 0 ? !p.io.w_post && !channel : !p.io.dw_pre) return;
    const int r0 = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
    const int64_t pitch = part_pitch(H);
    const float *at = p.part + which * pitch + col0 + c;   // the padding's columns are read and not used
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 5
    for (int r = r0; r < parts; r += kRows) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(at + r * 2 * pitch));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    sum[r0][c] = s.x, sum[r0][c + 1] = s.y, sum[r0][c + 2] = s.z, sum[r0][c + 3] = s.w;
    __syncthreads();
    constexpr int kWarps = kRows / 4;
#pragma unroll
    for (int k = warp; k < 32; k += kWarps) {
        float v = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; r += 32) v += sum[r + lane][k];
        v = warp_sum(v);
        const int out = col0 + k;
        if (lane != 0 || out >= H) continue;
        if (which == 1) {
            p.io.dw_pre[out] = v;
            continue;
        }
        if (p.io.w_post) p.io.dw_post[out] = channel ? v * load_param(p.io.gate, p.param_f32, out) : v;
        if (channel) p.io.dgate[out] = p.io.w_post ? v * load_param(p.io.w_post, p.param_f32, out) : v;
    }
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

bool rows16(const void *p, int64_t ld, size_t es) { return !p || (aligned_to(p, 16) && ld * es % 16 == 0); }

// Slots of a CTA that shares its SM with ctas - 1 others, `row` bytes each.
constexpr size_t kRingBytes = 216 * 1024;
int ring_slots(size_t row, int ctas, size_t params) {
    const size_t room = kRingBytes / ctas > params ? kRingBytes / ctas - params : 0;
    return (int)std::max<size_t>(1, std::min<size_t>(kMaxSlots, room / row));
}

template <class S, int NV, Map M, bool kWarpRow, Keep kKeep, int kMaxThreads, int kMinCtas>
cudaError_t launch_fwd(NormFwd p, cudaStream_t s) {
    const int per_thread = 8 * NV * 32;   // columns of a warp
    const int threads = kWarpRow ? 128 : (p.H + per_thread - 1) / per_thread * 32;
    const auto kernel = norm_fwd_kernel<S, NV, M, kWarpRow, kKeep, kMaxThreads, kMinCtas>;
    if (kWarpRow) return launch(kernel, ((unsigned)p.T + 3) / 4, threads, 0, 1, s, p);
    const int per_sm = std::max(1, kMaxThreads * kMinCtas / threads);
    size_t smem = 0;
    if (M == kVec) {
        const size_t row = (size_t)2 * NV * threads * 8 * sizeof(S);
        const size_t params = (size_t)2 * Params<NV, kKeep>::kBytes * threads;
        p.slots = ring_slots(row, per_sm, params);
        smem = p.slots * row + params;
        static std::atomic<uint32_t> done{0};
        const cudaError_t e = smem_limit_once((const void *)kernel, kRingBytes, done);
        if (e != cudaSuccess) return e;
    }
    return launch(kernel, std::min(p.T, 152 * per_sm), threads, smem, 1, s, p);
}

template <class S, Map M>
cudaError_t launch_fwd(const NormFwd &p, cudaStream_t s) {
    // A warp holds a short row without barriers (4096 x 512 bf16: 6.1 us, as CTAs of a warp that walk rows 9.6).  From 513
    // columns on, aligned rows are faster in CTAs that walk (32768 x 1024: 57.5 us, a row a warp 65.5; at 600 rows 5.3 and
    // 5.0); by element, where nothing is copied ahead, a warp still wins (4096 x 1001: 14.8 us against 35).
    if (p.H <= 256) return launch_fwd<S, 1, M, true, kNone, 128, 1>(p, s);
    if (p.H <= 512) return launch_fwd<S, 2, M, true, kNone, 128, 1>(p, s);
    if constexpr (M == kVec) {
        // More rows than SMs: two CTAs an SM, so that one works while the other waits at its barrier, with the parameters
        // in shared memory because no registers are left for them (4096 x 7168 bf16: 44.2 us, one CTA with registers 53.8;
        // 160 rows 6.2 and 6.1).  Fewer rows: each has an SM to itself, and registers save the trip (1 row 3.9 us against
        // 4.2, 128 rows 4.1 against 5.8).  f32 rows are twice as long, which leaves two CTAs' shared memory no second slot
        // beside the parameters: registers (1767 x 4096: 24.8 us against 29.1, 2000 x 7168 42.7 and 42.3).
        if constexpr (sizeof(S) == 2)
            if (p.H <= 8192 && p.T > 152) return launch_fwd<S, 2, M, false, kShared, 512, 2>(p, s);
    } else {
        if (p.H <= 1024) return launch_fwd<S, 4, M, true, kNone, 128, 1>(p, s);
    }
    if (p.H <= 8192) return launch_fwd<S, 2, M, false, kRegs, 512, 1>(p, s);
    return launch_fwd<S, 2, M, false, kNone, 1024, 1>(p, s);
}

template <class S>
cudaError_t launch_fwd_any(const NormFwd &p, cudaStream_t s) {
    const moe_norm_io &io = p.io;
    const size_t es = sizeof(S);
    const bool vec = p.H % 8 == 0 && rows16(io.residual, io.ld_residual, es) && rows16(io.y, io.ld_y, es) &&
                     rows16(io.h, io.ld_h, es) && rows16(io.n, io.ld_n, es) && aligned_to(io.w_post, 16) &&
                     aligned_to(io.w_pre, 16) && (p.gate != MOE_GATE_CHANNEL || aligned_to(io.gate, 16));
    if (vec) return launch_fwd<S, kVec>(p, s);
    return p.quant != MOE_QUANT_NONE ? launch_fwd<S, kChunk>(p, s) : launch_fwd<S, kStride>(p, s);
}

template <class S, int NV, int R, Map M, bool kWide, int kMaxThreads, int kMinCtas>
cudaError_t launch_bwd(NormBwd p, int parts, cudaStream_t s) {
    const int per_thread = 8 * NV * 32;
    const int threads = (p.H + per_thread - 1) / per_thread * 32;
    const auto kernel = norm_bwd_kernel<S, NV, R, M, kWide, kMaxThreads, kMinCtas>;
    const size_t params = (size_t)2 * Params<NV, bwd_keep(R, kWide)>::kBytes * threads;
    size_t smem = 0;
    if (kWide) {
        smem = (size_t)2 * NV * 8 * threads * 4;
    } else if (M == kVec) {
        const size_t row = (size_t)4 * R * NV * threads * 8 * sizeof(S);
        p.slots = ring_slots(row, std::max(1, kMaxThreads * kMinCtas / threads), params);
        smem = p.slots * row + params;
    }
    if (smem > 0) {
        static std::atomic<uint32_t> done{0};
        const cudaError_t e = smem_limit_once((const void *)kernel, kRingBytes, done);
        if (e != cudaSuccess) return e;
    }
    return launch(kernel, parts, threads, smem, 1, s, p);
}

// CTAs of the backward pass, `per_sm` on each SM, or the rows.
int ctas_of(int T, int per_sm) { return std::max(1, std::min(T, 152 * per_sm)); }

// CTAs an SM holds with two chunks a thread and 128 registers, or 64 (kWide).
int bwd_per_sm(int H, bool wide) { return std::max(1, std::min(8, (wide ? 1024 : 512) / ((H + 511) / 512 * 32))); }

// `parts`: the CTAs, each of which leaves a row of partial sums.
template <class S, Map M>
cudaError_t launch_bwd(const NormBwd &p, int &parts, cudaStream_t s) {
    if constexpr (M == kVec) {
        // Two rows a pass where both fit the CTA's shared memory: half the barriers, and the parameters read once for two
        // (4096 x 7168 bf16: 76 us, one row a pass 86).
        constexpr int kRows = sizeof(S) == 2 ? 2 : 1;
        const int per_sm = bwd_per_sm(p.H, false);
        // Few short rows, less than two passes a CTA: one chunk a thread and a row a pass (300 x 1024 bf16: 7.8 us against
        // 10.3; 32768 x 1024: 92 against 71).
        if (p.H <= 2048 && p.T < 2 * 152 * per_sm)
            return launch_bwd<S, 1, 1, M, false, 256, 2>(p, parts = ctas_of(p.T, p.H <= 1024 ? 4 : 2), s);
        // A row to a CTA: no second one (152 x 7168 bf16: 13.1 us, against 14.9; 1 x 4096: 7.5 and 9.2).
        if (p.H <= 8192 && (kRows == 1 || p.T <= 152 * per_sm))
            return launch_bwd<S, 2, 1, M, false, 512, 1>(p, parts = ctas_of(p.T, per_sm), s);
        if (p.H <= 8192) return launch_bwd<S, 2, kRows, M, false, 512, 1>(p, parts = ctas_of(p.T, per_sm), s);
        return launch_bwd<S, 2, 1, M, true, 1024, 1>(p, parts = ctas_of(p.T, 1), s);
    } else {
        // By element into registers a row ahead: one chunk a thread, for which they last.  Wider rows come in as they are
        // needed, behind other CTAs' (4096 x 5001 bf16: 193 us, two chunks a thread ahead, spilled, 281).
        if (p.H <= 2048) return launch_bwd<S, 1, 1, M, false, 256, 2>(p, parts = ctas_of(p.T, p.H <= 1024 ? 4 : 2), s);
        if (p.H <= 4096) return launch_bwd<S, 1, 1, M, false, 512, 1>(p, parts = ctas_of(p.T, 1), s);
        return launch_bwd<S, 2, 1, M, true, 1024, 1>(p, parts = ctas_of(p.T, bwd_per_sm(p.H, true)), s);
    }
}

// The most that launch_bwd takes.
int bwd_parts(int H, int T) { return ctas_of(T, bwd_per_sm(H, H > 4096)); }

template <class S>
cudaError_t launch_bwd_any(const NormBwd &p, int &parts, cudaStream_t s) {
    const moe_norm_grad_io &io = p.io;
    const size_t es = sizeof(S);
    const bool vec = p.H % 8 == 0 && rows16(io.h, io.ld_h, es) && rows16(io.y, io.ld_y, es) && rows16(io.dh, io.ld_dh, es) &&
                     rows16(io.dn, io.ld_dn, es) && rows16(io.dresidual, io.ld_dresidual, es) && rows16(io.dy, io.ld_dy, es) &&
                     aligned_to(io.w_post, 16) && aligned_to(io.w_pre, 16) &&
                     (p.gate != MOE_GATE_CHANNEL || aligned_to(io.gate, 16));
    return vec ? launch_bwd<S, kVec>(p, parts, s) : launch_bwd<S, kStride>(p, parts, s);
}

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
    NormFwd p{*io, num_tokens, H, io->w_pre ? cfg->quant : (int)MOE_QUANT_NONE, io->y ? cfg->gate : (int)MOE_GATE_NONE, 1,
              cfg->param_dtype == MOE_DTYPE_F32, cfg->eps, cfg->residual_scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cfg->stream_dtype == MOE_DTYPE_F32 ? launch_fwd_any<float>(p, s) : launch_fwd_any<bf16>(p, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_workspace_bytes(const moe_norm_config *cfg, int num_tokens) {
    if (!valid(cfg) || num_tokens < 0) return 0;
    const size_t b = (size_t)bwd_parts(cfg->hidden, num_tokens) * 2 * part_pitch(cfg->hidden) * 4;
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
    int parts = 0;
    NormBwd p{*io, static_cast<float *>(d_workspace), num_tokens, H, io->y ? cfg->gate : (int)MOE_GATE_NONE, 1,
              cfg->param_dtype == MOE_DTYPE_F32, cfg->residual_scale};
    const cudaError_t e = cfg->stream_dtype == MOE_DTYPE_F32 ? launch_bwd_any<float>(p, parts, s) : launch_bwd_any<bf16>(p, parts, s);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (sums) {
        const int ctas = 2 * ((H + 31) / 32);
        const cudaError_t e = parts > 256 ? launch(norm_bwd_sum_kernel<128>, ctas, 1024, 0, 1, s, p, parts)
                                          : launch(norm_bwd_sum_kernel<32>, ctas, 256, 0, 1, s, p, parts);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
