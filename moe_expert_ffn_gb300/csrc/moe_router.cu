// moe_router.cu -- the top-k router, the balance and z losses with per-sequence
// expert counts, and the gradient of the logits (definitions in
// include/moe.h).
//
// Large batches are bound by instructions, not by the [T, E] logits: one pass
// reads them once, and what counts is the choice.  A token belongs to a group
// of 32 lanes (8 for E <= 64), lane l holding experts l, l + G, ...: coalesced
// for any E and pitch.  Keys are made whole numbers: the float's order in the
// high bits, the expert, inverted, in the low ones.  So no two are equal, a
// lane sorts its keys with minima and maxima alone, and a round of the choice
// is one reduction over the lanes' heads, whose winner knows itself.  Whatever
// f32 bits the expert's number displaced can matter only where two
// neighbours in the result share all bits above (1 token in some hundreds;
// none with bf16 logits, which have no such bits): those are ranked anew by
// their full keys, or, at the edge of the chosen, the token is chosen again.
// (When every such token was chosen again, the few warps that met two of them
// held up the rest: 17 us for 32767 tokens whose average warp took 11.)
//
// Losses: CTAs walk contiguous token ranges, cut where a sequence ends; within
// a cut every lane sums its experts' probabilities in registers, the CTA's
// warps are joined in shared memory, and one row of partial sums is written.
// CTA b in sequence s uses row b + s: along the walk either one grows with
// every cut, so rows never collide, and the rows of a sequence are those of
// the consecutive CTAs that its tokens fall on.  All sums are taken in a fixed
// order: no float atomics, the same bits every time.
//
// Measured: 32767 tokens of 256 bf16 logits, 8 chosen, sigmoid with a bias:
// 18.5 us, 380 warp instructions a token, two thirds of the issue slots taken
// and the integer pipe the busiest (reading the logits alone would take 2.8; a
// simple kernel 38.9).  65536 tokens of 256 f32 logits in 17 sequences with
// losses and the whole gradient: 77 us (forward 40, sums 5, backward 32; bytes
// alone 21.1; simple kernels 339).  128 tokens: 2.0 us.  2048 tokens of 8
// experts, losses of a given choice and gradient: 8.0 us, three launches,
// each a chain of a few trips to memory.
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
constexpr int kMaxCtas = 608;   // four on each of 152 SMs
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.44269504f;

// Rows of partial sums and what follows them in the workspace.
struct Partials {
    float *prob;      // [rows][E]
    int32_t *count;   // [rows][E]
    float *z;         // [rows]
    int32_t *tokens;  // [rows]
    float *seq_bal;   // [S][E / 32]
    float *seq_z;     // [S]
    int *ticket;
};

struct RouterParams {
    const void *logits;
    int64_t ld;
    const float *bias;
    int32_t *topk_idx;          // out, or in with kGiven
    float *topk_weights;
    const int32_t *seq_offsets;
    Partials part;
    int T, E, k, S, chunk;      // chunk: tokens per CTA
    int sigmoid, renorm, score_bias;
    float scale;
};

// A logit as it enters choice and scores: NaN and -inf are closed (-inf), +inf is the largest float.
__device__ __forceinline__ float open_logit(float v) { return fminf(fmaxf(v, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float exp2_of(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// e^v: its relative error is that of the rounded exponent, 2^-24 of |v| log2(e), plus 2 units in the last place.
__device__ __forceinline__ float exp_of(float v) { return exp2_of(v * kLog2e); }

// Sigmoid times e^-m with m = min(largest logit, 0): the ratios of the scores of a token whose sigmoids all underflow
// stay right.
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
    const float u = exp_of(-fabsf(l));
    const float d = __fdividef(1.0f, 1.0f + u);
    return l >= 0.0f ? d : (m < 0.0f ? exp_of(l - m) : u) * d;
}
// sigmoid(l), -inf where closed.  With the losses as a call of its own: in line it takes registers from the passes that do
// not use it (65536 x 256 losses and gradient 77.9 us, 76.9 with the call; without losses 20.5 in line, 23.2).
__device__ __forceinline__ float score_of(float l) { return l > -INFINITY ? sigmoid_scaled(l, 0.0f) : -INFINITY; }
__device__ __noinline__ float score_of_call(float l) { return score_of(l); }
// 1 - sigmoid(l)
__device__ __forceinline__ float sigmoid_slope(float l) {
    const float u = exp_of(-fabsf(l));
    return (l >= 0.0f ? u : 1.0f) * __fdividef(1.0f, 1.0f + u);
}

// Reductions over the G lanes of a token; every lane gets the result.
template <int G>
__device__ __forceinline__ float group_max(float v) {
    if (G == 32) {
        float r;
        asm("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(kAll));
        return r;
    }
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ int group_min(int v) {
    if (G == 32) return __reduce_min_sync(kAll, v);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// The first s in [s0, S) with off[s + 1] > t, else S; every lane of a warp calls and gets it.  One load asks for 32
// offsets: the next ones, where a walk's sequences are, then those that cut the rest into 32.  (A search by halves, anew
// for every cut, made most of the time of small batches: 19 tokens in 20 sequences 56 us for losses and gradient.)
__device__ __forceinline__ int find_seq(const int32_t *off, int S, int t, int s0) {
    const int lane = threadIdx.x & 31;
    int lo = s0, hi = S, step = 1;   // the answer is in [lo, hi]; hi is S or was seen to end past t
    while (lo < hi) {
        const int m = lo + (lane + 1) * step - 1;
        const unsigned past = __ballot_sync(kAll, m < hi && off[m + 1] > t);
        if (past) {
            const int f = __ffs(past) - 1;
            hi = lo + (f + 1) * step - 1;
            lo += f * step;
        } else {
            lo += min(32, (hi - lo) / step) * step;
        }
        step = (hi - lo + 31) / 32;
    }
    return hi;
}

// The sequence (or the gap before it) that token t is in, from sequence s0 on: its index, whether it counts, and where
// the cut ends.
struct Cut {
    int s, end;
    bool inside;
};
__device__ __forceinline__ Cut cut_at(const int32_t *off, int S, int t, int t1, int s0) {
    Cut c{0, t1, true};
    if (!off) return c;
    c.s = find_seq(off, S, t, s0);
    if (c.s >= S) return Cut{S, t1, false};
    const int begin = off[c.s], end = off[c.s + 1];
    c.inside = t >= begin;
    c.end = min(t1, c.inside ? end : begin);
    return c;
}

// A token's logits as loaded (-inf where there is none), so that the next token's can be on their way.
template <class L, int NI, int G>
__device__ __forceinline__ void load_row(L (&l)[NI], const void *logits, int64_t ld, uint32_t t, bool on, int lg, int E) {
    const L *row = static_cast<const L *>(logits) + (int64_t)t * ld + lg;
    if (E == NI * G) {   // every lane has all its experts
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = on ? row[G * i] : from_f32<L>(-INFINITY);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = on && lg + G * i < E ? row[G * i] : from_f32<L>(-INFINITY);
    }
}

// Logits as the definitions take them (open_logit): needed only where a NaN or +inf turns up, which the callers see in
// what they compute.
template <int NI>
__device__ __forceinline__ void clean(float (&l)[NI]) {
#pragma unroll
    for (int i = 0; i < NI; ++i) l[i] = open_logit(l[i]);
}

// Scores of a token's logits times e^-(m or min(m, 0)), 0 where closed, and their sum.  Cleans l and m if need be.
template <int NI, int G>
__device__ __forceinline__ float scores(float (&q)[NI], float (&l)[NI], float &m, bool sigmoid) {
    float z = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        z = 0.0f;
        if (sigmoid) {
            const float ms = fminf(m, 0.0f);
#pragma unroll
            for (int i = 0; i < NI; ++i) z += q[i] = sigmoid_scaled(l[i], ms);
        } else {
            if (NI % 2 == 0) {
                float2 zz = pair(0.0f);
#pragma unroll
                for (int i = 0; i + 1 < NI; i += 2) {
                    const float2 v = __fmul2_rn(__fadd2_rn(make_float2(l[i], l[i + 1]), pair(-m)), pair(kLog2e));
                    q[i] = exp2_of(v.x), q[i + 1] = exp2_of(v.y);
                    zz = __fadd2_rn(zz, make_float2(q[i], q[i + 1]));
                }
                z = zz.x + zz.y;
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) z += q[i] = exp_of(l[i] - m);
            }
        }
        z = group_sum<G>(z);
        if (!__any_sync(kAll, !(z <= FLT_MAX))) break;
        clean(l);
        m = fminf(m, FLT_MAX);
    }
    return z;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if (G == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Sorts in descending order by compare-exchanges (merge-exchange network for NI a power of two).
template <int NI>
__device__ __forceinline__ void sort_down(uint32_t (&v)[NI]) {
#pragma unroll
    for (int p = NI / 2; p > 0; p /= 2) {
#pragma unroll
        for (int q = NI / 2, r = 0, d = p; d > 0; d = q - p, q /= 2, r = p) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (i + d < NI && (i & p) == r) {
                    const uint32_t a = v[i], b = v[i + d];
                    v[i] = max(a, b);
                    v[i + d] = min(a, b);
                }
            if (q < p) break;
        }
    }
}

__device__ __forceinline__ void exchange(uint32_t &a, uint32_t &b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// The D largest of v, descending, in v[0..D): all of them, or 4 by sorting fours and merging.
template <int NI, int D>
__device__ __forceinline__ void top_down(uint32_t (&v)[NI]) {
    if (D == NI) {
        sort_down(v);
        return;
    }
#pragma unroll
    for (int b = 0; b < NI; b += 4) {
        exchange(v[b], v[b + 1]);
        exchange(v[b + 2], v[b + 3]);
        exchange(v[b], v[b + 2]);
        exchange(v[b + 1], v[b + 3]);
        exchange(v[b + 1], v[b + 2]);
    }
#pragma unroll
    for (int w = 4; w < NI; w *= 2)
#pragma unroll
        for (int b = 0; b < NI; b += 2 * w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[b + i] = max(v[b + i], v[b + w + 3 - i]);   // the 4 largest of both, bitonic
            exchange(v[b], v[b + 2]);
            exchange(v[b + 1], v[b + 3]);
            exchange(v[b], v[b + 1]);
            exchange(v[b + 2], v[b + 3]);
        }
}

// The k largest keys of a group's token from the full keys, one by one: the exact choice whatever the keys.
template <int NI, int G, int NS>
__device__ __noinline__ void choose_exact(const float (&key)[NI], int k, int lg, int (&slot_e)[NS]) {
    uint32_t taken = 0;
#pragma unroll
    for (int q = 0; q < NS; ++q) slot_e[q] = -1;
    for (int j = 0; j < k; ++j) {
        float best = -INFINITY;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (!((taken >> i) & 1) && key[i] > best) best = key[i], bi = i;   // of equal keys the first stays
        const float m = group_max<G>(best);
        int e = group_min<G>(best == m && m > -INFINITY ? lg + G * bi : 1 << 20);
        if (e < 1 << 20) {
            if ((e & (G - 1)) == lg) taken |= 1u << (e / G);
        } else {
            e = -1;
        }
#pragma unroll
        for (int q = 0; q < NS; ++q)
            if (j == q * G + lg) slot_e[q] = e;
    }
}

// The k largest keys of a group's token, ties to the lowest expert.  Slot j goes to lane j % G, place j / G: its expert
// (-1: nothing left).  `exact`: the keys' low bits that the expert's number takes say nothing.  A lane keeps its D
// largest; one that wins D < NI times may have had more.  Returns false, with nothing chosen, where a key is +inf or a
// NaN that sorts above it and `cleaned` does not say that it is meant.
template <int NI, int G, int NS, int D>
__device__ __forceinline__ bool choose(const float (&key)[NI], int k, int lg, bool exact, bool cleaned, int (&slot_e)[NS]) {
    constexpr uint32_t kLow = (uint32_t)(NI * G - 1);   // bits of an expert's number
    constexpr uint32_t kOpen = 0x00800000u;             // the order of the smallest finite float
    auto packed = [&](int i) {
        const uint32_t b = __float_as_uint(key[i] + 0.0f);   // -0 and 0 are equal
        const uint32_t order = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
        return (order & ~kLow) | (kLow - (uint32_t)(lg + G * i));
    };
    uint32_t v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = packed(i);
    top_down<NI, D>(v);
    if (!cleaned && __any_sync(kAll, v[0] >= 0xFF800000u)) return false;   // the order of +inf
    uint32_t slot[NS], last = 0;
#pragma unroll
    for (int q = 0; q < NS; ++q) slot[q] = 0;
    for (int j = 0; j < k; ++j) {
        last = group_max<G>(v[0]);
#pragma unroll
        for (int q = 0; q < NS; ++q)
            if (j == q * G + lg) slot[q] = last;
        const bool won = v[0] == last;
#pragma unroll
        for (int i = 0; i + 1 < D; ++i) v[i] = won ? v[i + 1] : v[i];
        v[D - 1] = won ? 0u : v[D - 1];
    }
    bool again = false;
    if (D < NI && __any_sync(kAll, v[0] == 0)) {   // a lane gave all it kept: had it more that belong?
        // one that it did not keep may share the last one's high bits and have the larger full key; closed ones do not count
        const uint32_t least = max(exact ? last : last & ~kLow, kOpen);
        int n = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) n += packed(i) >= least;
        again = n > D;
    }
#pragma unroll
    for (int q = 0; q < NS; ++q) slot_e[q] = slot[q] < kOpen ? -1 : (int)(kLow - (slot[q] & kLow));
    if (!exact) {   // open neighbours that only the displaced bits tell apart, among the chosen and at their edge
        const uint32_t out = group_max<G>(v[0]);
        bool near = false;
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            uint32_t next = __shfl_down_sync(kAll, slot[q], 1, G);
            const uint32_t wrap = __shfl_sync(kAll, slot[q + 1 < NS ? q + 1 : q], 0, G);
            if (lg == G - 1) next = q + 1 < NS ? wrap : out;
            const bool edge = q * G + lg == k - 1;
            if (edge) next = out;
            const bool same = q * G + lg < k && slot[q] >= kOpen && ((slot[q] ^ next) & ~kLow) == 0;
            near |= same && !edge;
            again |= same && (edge || NS > 1);
        }
        if (NS == 1 && __any_sync(kAll, near) && !__any_sync(kAll, again)) {
            // the right ones in a wrong order: ranked anew by their full keys
            const int e = lg < k ? slot_e[0] : -1;
            float mine = -INFINITY;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float f = __shfl_sync(kAll, key[i], e & (G - 1), G);
                if (e >= 0 && e / G == i) mine = f;
            }
            int rank = 0;   // empty slots (e = -1) stay behind all others
            for (int j = 0; j < k; ++j) {
                const float f = __shfl_sync(kAll, mine, j, G);
                const int fe = __shfl_sync(kAll, e, j, G);
                rank += f > mine || (f == mine && fe >= 0 && fe < e);
            }
            const int held = e;
            for (int j = 0; j < k; ++j) {
                const int r = __shfl_sync(kAll, rank, j, G), fe = __shfl_sync(kAll, held, j, G);
                if (fe >= 0 && r == lg) slot_e[0] = fe;
            }
        }
    }
    if (__any_sync(kAll, again)) choose_exact<NI, G, NS>(key, k, lg, slot_e);
    return true;
}

// Joins the warps of the CTA: sum of `v` over the groups of every warp, in warp order, for the lanes' experts.
template <int G>
__device__ __forceinline__ float over_groups(float v) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// CTAs an SM by the experts of a lane: what registers allow without spills that cost (32767 x 256: four 18.5 us, five or
// six 20.6 to 22; 28219 x 259: two 20.4, one 29.2).
constexpr int ctas_an_sm(int NI) { return NI <= 8 ? 4 : NI == 16 ? 2 : 1; }

template <class L, int NI, int G, int D, bool kLoss, bool kGiven>
__global__ void __launch_bounds__(kThreads, ctas_an_sm(NI)) router_kernel(const __grid_constant__ RouterParams p) {
    extern __shared__ float joined[];   // kLoss: [warps][E] probabilities, [E] counts
    __shared__ float sz[kWarps];
    __shared__ int sn[kWarps];
    constexpr int kGroups = 32 / G;                      // tokens of a warp at a time
    constexpr int NS = G == 32 ? 1 : 32 / G;             // slots of a lane (k <= 32)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), grp = lane / G;
    const int E = p.E, k = p.k;
    int *counts = reinterpret_cast<int *>(joined + kWarps * E);
    const int t0 = (int)min((int64_t)blockIdx.x * p.chunk, (int64_t)p.T), t1 = (int)min((int64_t)t0 + p.chunk, (int64_t)p.T);
    launch_next();
    wait_for_previous();
    if (kLoss && blockIdx.x == 0 && threadIdx.x == 0) *p.part.ticket = 0;   // for the next kernel
    float bias[NI];
    if (!kGiven && p.bias) {
#pragma unroll
        for (int i = 0; i < NI; ++i) bias[i] = lg + G * i < E ? p.bias[lg + G * i] : 0.0f;
    }
    int s_at = 0;
    for (int a = t0; a < t1;) {
        const Cut cut = kLoss ? cut_at(p.seq_offsets, p.S, a, t1, s_at) : Cut{0, t1, true};
        s_at = cut.s;
        L raw[NI];
        const uint32_t end = cut.end, tw = (uint32_t)a + warp * kGroups;   // a step past the last token may pass 2^31
        if (tw < end) load_row<L, NI, G>(raw, p.logits, p.ld, tw + grp, tw + grp < end, lg, E);
        float prob[kLoss ? NI : 1];
        float zsum = 0.0f;
        int tokens = 0;
        if (kLoss) {
#pragma unroll
            for (int i = 0; i < NI; ++i) prob[i] = 0.0f;
            for (int e = threadIdx.x; e < E; e += kThreads) counts[e] = 0;
            __syncthreads();
        }
        for (uint32_t tb = tw; tb < end; tb += kWarps * kGroups) {
            const uint32_t t = tb + grp;
            const bool on = t < end;
            float l[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) l[i] = to_f32(raw[i]);
            const uint32_t tn = tb + kWarps * kGroups;
            if (tn < end) load_row<L, NI, G>(raw, p.logits, p.ld, tn + grp, tn + grp < end, lg, E);
            float m = -INFINITY, top = -INFINITY;   // the largest logit, and that of the chosen
            if (kGiven || (kLoss && p.bias) || (!p.renorm && !p.sigmoid)) {
#pragma unroll
                for (int i = 0; i < NI; ++i) m = fmaxf(m, l[i]);
                m = fminf(group_max<G>(m), FLT_MAX);
            }
            int my_e[NS];
            if (kGiven) {
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const int j = q * G + lg;
                    my_e[q] = on && j < k ? p.topk_idx[(int64_t)t * k + j] : -1;
                    if (my_e[q] >= E) my_e[q] = -1;
                }
            } else {
                for (int pass = 0; pass < 2; ++pass) {
                    float key[NI];
#pragma unroll
                    for (int i = 0; i < NI; ++i) key[i] = l[i];
                    if (p.score_bias) {   // 32767 x 256 bf16 20.5 us, on the logits 18.3
#pragma unroll
                        for (int i = 0; i < NI; ++i) key[i] = kLoss ? score_of_call(l[i]) : score_of(l[i]);
                    }
                    if (p.bias) {
#pragma unroll
                        for (int i = 0; i < NI; ++i) key[i] += bias[i];
                    }
                    if (pass) {   // -inf + inf closes
#pragma unroll
                        for (int i = 0; i < NI; ++i) key[i] = fmaxf(key[i], -INFINITY);
                    }
                    if (choose<NI, G, NS, D>(key, k, lg, sizeof(L) == 2 && !p.bias, pass, my_e)) break;
                    clean(l);
                }
                // weights of the chosen
                float wgt[NS], my_l[NS], f = p.scale;
#pragma unroll
                for (int q = 0; q < NS; ++q)
                    my_l[q] = my_e[q] < 0 ? -INFINITY
                                          : open_logit(to_f32(static_cast<const L *>(p.logits)[(int64_t)t * p.ld + my_e[q]]));
                if (p.renorm || kLoss) {
#pragma unroll
                    for (int q = 0; q < NS; ++q) top = fmaxf(top, my_l[q]);
                    top = group_max<G>(top);
                    if (kLoss && !p.bias) m = top;
                }
                if (p.renorm) {
                    float sum = 0.0f;
#pragma unroll
                    for (int q = 0; q < NS; ++q) {
                        wgt[q] = my_e[q] < 0 ? 0.0f : p.sigmoid ? sigmoid_scaled(my_l[q], fminf(top, 0.0f)) : exp_of(my_l[q] - top);
                        sum += wgt[q];
                    }
                    sum = group_sum<G>(sum);
                    f = sum > 0.0f ? __fdividef(f, sum) : 0.0f;
                } else if (p.sigmoid) {
#pragma unroll
                    for (int q = 0; q < NS; ++q) wgt[q] = my_e[q] < 0 ? 0.0f : sigmoid_scaled(my_l[q], 0.0f);
                } else {
                    float all[NI];
                    float m0 = m > -INFINITY ? m : 0.0f;
                    const float sum = scores<NI, G>(all, l, m0, false);
                    f = sum > 0.0f ? __fdividef(f, sum) : 0.0f;
#pragma unroll
                    for (int q = 0; q < NS; ++q) wgt[q] = my_e[q] < 0 ? 0.0f : exp_of(my_l[q] - m0);
                }
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const int j = q * G + lg;
                    if (on && j < k) {
                        p.topk_idx[(int64_t)t * k + j] = my_e[q];
                        p.topk_weights[(int64_t)t * k + j] = wgt[q] * f;
                    }
                }
            }
            if (kLoss && cut.inside) {
                const bool real = m > -INFINITY;
                float q[NI];
                m = real ? m : 0.0f;
                const float z = scores<NI, G>(q, l, m, p.sigmoid);
                const float inv = real ? __fdividef(1.0f, z) : 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) prob[i] = fmaf(q[i], inv, prob[i]);
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (real && my_e[s] >= 0) atomicAdd(counts + my_e[s], 1);   // whole numbers: the order does not matter
                if (real && lg == 0) {
                    const float lse = m + __logf(z);   // z >= 1
                    zsum += p.sigmoid ? 0.0f : lse * lse;
                    ++tokens;
                }
            }
        }
        if (kLoss) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lg + G * i;
                const float pr = over_groups<G>(prob[i]);
                if (e < E && grp == 0) joined[warp * E + e] = pr;
            }
            zsum = warp_sum(zsum);
            tokens = __reduce_add_sync(kAll, tokens);
            if (lane == 0) sz[warp] = zsum, sn[warp] = tokens;
            __syncthreads();
            const int64_t row = (int64_t)blockIdx.x + cut.s;
            for (int e = threadIdx.x; e < E; e += kThreads) {
                float pr = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) pr += joined[w * E + e];
                p.part.prob[row * E + e] = pr;
                p.part.count[row * E + e] = counts[e];
            }
            if (threadIdx.x == 0) {
                float z = 0.0f;
                int n = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) z += sz[w], n += sn[w];
                p.part.z[row] = z;   // a gap before sequence s writes zeros where s, if it starts in this CTA, writes next
                p.part.tokens[row] = n;
            }
            __syncthreads();
        }
        a = cut.end;
    }
}

struct SumParams {
    Partials part;
    const int32_t *seq_offsets;
    int32_t *counts;
    float *prob_mean;
    int32_t *seq_tokens;
    float *loss;
    int T, E, k, S, chunk;
    float alpha, beta;
};

// CTA (s, x): 32 experts of sequence s, its rows summed in order (a thread takes every W-th row, then the W are added in
// turn).  The last CTA to finish adds up the losses.
template <int W>
__global__ void __launch_bounds__(W * 32) router_seq_kernel(const __grid_constant__ SumParams p) {
    __shared__ float sp[W][32];
    __shared__ int sc[W][32];
    __shared__ float sz[W];
    __shared__ int sn[W];
    __shared__ bool last;
    launch_next();
    const int slabs = (p.E + 31) / 32, s = blockIdx.x / slabs, slab = blockIdx.x - s * slabs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = slab * 32 + lane;
    wait_for_previous();
    const int a = p.seq_offsets ? max(0, min(p.seq_offsets[s], p.T)) : 0;
    const int b = p.seq_offsets ? max(0, min(p.seq_offsets[s + 1], p.T)) : p.T;
    const int w0 = a / p.chunk, w1 = b > a ? (b - 1) / p.chunk + 1 : w0;
    float pr = 0.0f, z = 0.0f;
    int c = 0, n = 0;
#pragma unroll 4
    for (int w = w0 + warp; w < w1; w += W)
        if (e < p.E) {
            pr += p.part.prob[(int64_t)(w + s) * p.E + e];
            c += p.part.count[(int64_t)(w + s) * p.E + e];
        }
    for (int w = w0 + threadIdx.x; w < w1; w += W * 32) {
        n += p.part.tokens[w + s];
        z += p.part.z[w + s];
    }
    sp[warp][lane] = pr;
    sc[warp][lane] = c;
    z = warp_sum(z);
    n = __reduce_add_sync(kAll, n);
    if (lane == 0) sz[warp] = z, sn[warp] = n;
    __syncthreads();
    if (warp == 0) {
        pr = 0.0f, z = 0.0f, c = 0, n = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) pr += sp[w][lane], c += sc[w][lane], z += sz[w], n += sn[w];
        const float mean = n > 0 ? pr / (float)n : 0.0f;
        if (e < p.E) {
            p.counts[(int64_t)s * p.E + e] = c;
            p.prob_mean[(int64_t)s * p.E + e] = mean;
        }
        const float bal = warp_sum(e < p.E ? (float)c * mean : 0.0f);
        if (lane == 0) {
            p.part.seq_bal[blockIdx.x] = n > 0 ? bal * (float)p.E / ((float)p.k * (float)n) : 0.0f;
            if (slab == 0) p.seq_tokens[s] = n, p.part.seq_z[s] = z;
            last = gridDim.x == 1;   // alone, it reads what this thread wrote
            if (!last) {
                __threadfence();
                last = atomicAdd(p.part.ticket, 1) == (int)gridDim.x - 1;
            }
        }
    }
    __syncthreads();
    if (!last || warp != 0) return;
    __threadfence();
    float bal = 0.0f;
    int used = 0;
    z = 0.0f, n = 0;
    for (int i = lane; i < (int)gridDim.x; i += 32) bal += __ldcg(p.part.seq_bal + i);
    for (int i = lane; i < p.S; i += 32) {
        const int ns = __ldcg(p.seq_tokens + i);
        z += __ldcg(p.part.seq_z + i);
        used += ns > 0;
        n += ns;
    }
    bal = warp_sum(bal);
    z = warp_sum(z);
    used = __reduce_add_sync(kAll, used);
    n = __reduce_add_sync(kAll, n);
    if (lane == 0) {
        bal = used > 0 ? p.alpha * bal / (float)used : 0.0f;
        z = n > 0 ? p.beta * z / (float)n : 0.0f;
        p.loss[0] = bal + z;
        p.loss[1] = bal;
        p.loss[2] = z;
        p.seq_tokens[p.S] = used;
        p.seq_tokens[p.S + 1] = n;
    }
}

struct RouterBwd {
    const void *logits;
    int64_t ld;
    const int32_t *topk_idx;
    const float *d_weights;
    const int32_t *seq_offsets, *counts, *seq_tokens;
    const float *d_loss;
    void *d_logits;
    int64_t ld_d;
    int T, E, k, S, chunk, sigmoid, renorm;
    float scale, alpha, beta;
};

template <class L, int NI, int G>
__global__ void __launch_bounds__(kThreads, ctas_an_sm(NI)) router_bwd_kernel(const __grid_constant__ RouterBwd p) {
    extern __shared__ float scatter[];   // [warps][groups][E]: gradients of the chosen logits, zero between tokens
    constexpr int kGroups = 32 / G;
    constexpr int NS = G == 32 ? 1 : 32 / G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane & (G - 1), grp = lane / G;
    const int E = p.E, k = p.k;
    float *mine = scatter + (warp * kGroups + grp) * E;
    launch_next();
    wait_for_previous();
    if (p.d_weights)
        for (int e = lg; e < E; e += G) mine[e] = 0.0f;
    __syncwarp();
    const int t0 = (int)min((int64_t)blockIdx.x * p.chunk, (int64_t)p.T), t1 = (int)min((int64_t)t0 + p.chunk, (int64_t)p.T);
    int s_at = 0;
    for (int a = t0; a < t1;) {
        const Cut cut = cut_at(p.seq_offsets, p.S, a, t1, s_at);
        s_at = cut.s;
        L raw[NI];
        int next_idx[NS];
        float next_dw[NS];
        auto load_slots = [&](uint32_t t, bool on) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int j = s * G + lg;
                next_idx[s] = on && j < k ? p.topk_idx[(int64_t)t * k + j] : -1;
                next_dw[s] = on && j < k ? p.d_weights[(int64_t)t * k + j] : 0.0f;
            }
        };
        const uint32_t end = cut.end, tw = (uint32_t)a + warp * kGroups;   // a step past the last token may pass 2^31
        if (tw < end) {
            load_row<L, NI, G>(raw, p.logits, p.ld, tw + grp, tw + grp < end, lg, E);
            if (p.d_weights) load_slots(tw + grp, tw + grp < end);
        }
        int n = 0;
        float c[NI], zc = 0.0f;   // the balance loss's pull on each expert's probability, the z loss's on log-sum-exp
        if (p.d_loss && cut.inside && cut.s < p.S) {
            int count[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) count[i] = lg + G * i < E ? p.counts[(int64_t)cut.s * E + lg + G * i] : 0;
            const float g = *p.d_loss, seqs = (float)p.seq_tokens[p.S], all = (float)p.seq_tokens[p.S + 1];
            n = p.seq_tokens[cut.s];
            const float c0 = n > 0 ? g * p.alpha * (float)E / ((float)k * (float)n * (float)n * seqs) : 0.0f;
            zc = p.sigmoid || n == 0 ? 0.0f : g * 2.0f * p.beta / all;
#pragma unroll
            for (int i = 0; i < NI; ++i) c[i] = c0 * (float)count[i];
        }
        const bool dense = n > 0 || (p.d_weights && !p.renorm && !p.sigmoid);   // every probability is needed
        for (uint32_t tb = tw; tb < end; tb += kWarps * kGroups) {
            const uint32_t t = tb + grp;
            const bool on = t < end;
            float l[NI], d[NI], q[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) l[i] = to_f32(raw[i]);
            const uint32_t tn = tb + kWarps * kGroups;
            if (tn < end) load_row<L, NI, G>(raw, p.logits, p.ld, tn + grp, tn + grp < end, lg, E);
            // the chosen slots' part
            float add[NS], ls[NS], dw[NS], dot = 0.0f;
            int idx[NS];
            if (p.d_weights) {
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    idx[s] = next_idx[s] < E ? next_idx[s] : -1;
                    ls[s] = idx[s] < 0 ? -INFINITY
                                       : open_logit(to_f32(static_cast<const L *>(p.logits)[(int64_t)t * p.ld + idx[s]]));
                    dw[s] = ls[s] > -INFINITY ? next_dw[s] * p.scale : 0.0f;   // a closed expert's may be anything
                }
                if (tn < end) load_slots(tn + grp, tn + grp < end);
            }
            float m = 0.0f, inv = 0.0f;
            bool real = false;
            if (dense) {
                m = -INFINITY;
#pragma unroll
                for (int i = 0; i < NI; ++i) m = fmaxf(m, l[i]);
                m = fminf(group_max<G>(m), FLT_MAX);
                real = m > -INFINITY;
                m = real ? m : 0.0f;
                const float z = scores<NI, G>(q, l, m, p.sigmoid);
                inv = real ? __fdividef(1.0f, z) : 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) q[i] *= inv;
                if (n > 0) {
                    const float lse = real ? m + __logf(z) : 0.0f;   // z >= 1 (sigmoid: unused)
                    float cq = 0.0f;
#pragma unroll
                    for (int i = 0; i < NI; ++i) cq = fmaf(c[i], q[i], cq);
                    cq = zc * lse - group_sum<G>(cq);
#pragma unroll
                    for (int i = 0; i < NI; ++i) d[i] = q[i] * (c[i] + cq);
                    if (p.sigmoid) {   // ds/dl = s (1 - s)
#pragma unroll
                        for (int i = 0; i < NI; ++i) d[i] *= sigmoid_slope(l[i]);
                    }
                }
            }
            if (n == 0) {
#pragma unroll
                for (int i = 0; i < NI; ++i) d[i] = 0.0f;
            }
            if (p.d_weights) {
                if (p.renorm) {
                    float top = -INFINITY, sum = 0.0f, mean = 0.0f;
#pragma unroll
                    for (int s = 0; s < NS; ++s) top = fmaxf(top, ls[s]);
                    top = group_max<G>(top);
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        add[s] = !(ls[s] > -INFINITY) ? 0.0f
                                 : p.sigmoid        ? sigmoid_scaled(ls[s], fminf(top, 0.0f))
                                                    : exp_of(ls[s] - top);
                        sum += add[s];
                    }
                    sum = group_sum<G>(sum);
                    const float r = sum > 0.0f ? __fdividef(1.0f, sum) : 0.0f;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        add[s] *= r;
                        mean = fmaf(add[s], dw[s], mean);
                    }
                    mean = group_sum<G>(mean);
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        add[s] *= dw[s] - mean;
                        if (p.sigmoid && ls[s] > -INFINITY) add[s] *= sigmoid_slope(ls[s]);
                    }
                } else if (p.sigmoid) {
#pragma unroll
                    for (int s = 0; s < NS; ++s)
                        add[s] = ls[s] > -INFINITY ? sigmoid_scaled(ls[s], 0.0f) * sigmoid_slope(ls[s]) * dw[s] : 0.0f;
                } else {
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        add[s] = real && ls[s] > -INFINITY ? exp_of(ls[s] - m) * inv * dw[s] : 0.0f;
                        dot += add[s];
                    }
                    dot = group_sum<G>(dot);
#pragma unroll
                    for (int i = 0; i < NI; ++i) d[i] = fmaf(-q[i], dot, d[i]);
                }
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (idx[s] >= 0) mine[idx[s]] = add[s];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (E == NI * G || lg + G * i < E) d[i] += mine[lg + G * i];
                __syncwarp();
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (idx[s] >= 0) mine[idx[s]] = 0.0f;
            }
            L *out = static_cast<L *>(p.d_logits) + (int64_t)t * p.ld_d + lg;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (on && (E == NI * G || lg + G * i < E)) out[G * i] = from_f32<L>(d[i]);
            __syncwarp();
        }
        a = cut.end;
    }
}

bool valid(const moe_router_config *c) {
    if (!c || c->num_experts < 1 || c->num_experts > 1024) return false;
    if (c->topk < 1 || c->topk > 32 || c->topk > c->num_experts) return false;
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return false;
    if (!valid_dtype(c->logits_dtype)) return false;
    if (!isfinite(c->weight_scale) || !isfinite(c->balance_coef) || !isfinite(c->z_coef)) return false;
    if (c->bias_on != MOE_BIAS_LOGIT && (c->bias_on != MOE_BIAS_SCORE || c->score != MOE_SCORE_SIGMOID)) return false;
    return c->score == MOE_SCORE_SOFTMAX || c->z_coef == 0.0f;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// CTAs of a pass over T tokens in S sequences, each with a contiguous part: no more than give every warp a turn, but eight
// to a sequence, because a CTA takes its sequences' parts one after the other (11 tokens in 5 sequences, losses and
// gradient: 8.6 us, with two to a sequence 10.8).
int ctas_for(int T, int E, int S) {
    const int per_cta = kWarps * (E <= 64 ? 4 : 1);
    const int even = (std::max(T, 1) - 1) / per_cta + 1;
    return std::min(std::max(even, S > 1 ? (int)std::min<int64_t>(T, (int64_t)8 * S) : 1), kMaxCtas);
}

// Carves the workspace; returns its size.
size_t carve(int E, int T, int S, char *base, Partials *out) {
    const size_t rows = (size_t)ctas_for(T, E, S) + S;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char *at = base + o;
        o += up256(bytes);
        return at;
    };
    Partials p;
    p.prob = reinterpret_cast<float *>(take(rows * E * 4));
    p.count = reinterpret_cast<int32_t *>(take(rows * E * 4));
    p.z = reinterpret_cast<float *>(take(rows * 4));
    p.tokens = reinterpret_cast<int32_t *>(take(rows * 4));
    p.seq_bal = reinterpret_cast<float *>(take((size_t)S * ((E + 31) / 32) * 4));
    p.seq_z = reinterpret_cast<float *>(take((size_t)S * 4));
    p.ticket = reinterpret_cast<int *>(take(4));
    if (out) *out = p;
    return o;
}

template <class L, int NI, int G, int D>
cudaError_t launch_router(const RouterParams &p, bool loss, int ctas, cudaStream_t s) {
    const size_t smem = (size_t)(kWarps + 1) * p.E * 4;   // at most 36 KB
    if (loss) return launch(router_kernel<L, NI, G, D, true, false>, ctas, kThreads, smem, 1, s, p);
    return launch(router_kernel<L, NI, G, D, false, false>, ctas, kThreads, 0, 1, s, p);
}
template <class L, int NI, int G>
cudaError_t launch_router(const RouterParams &p, bool loss, bool given, int ctas, cudaStream_t s) {
    if (given)
        return launch(router_kernel<L, NI, G, NI, true, true>, ctas, kThreads, (size_t)(kWarps + 1) * p.E * 4, 1, s, p);
    // up to 12 choices seldom fall four times on one of 32 lanes (1 token in 100 with 12), and four are cheaper to keep
    // in order than 8 and more (32767 tokens of 256 bf16: 12 chosen 22.4 us against 24.6, 8 chosen 18.8 against 20.4)
    constexpr int kFew = G == 32 && NI > 4 ? 4 : NI;
    if (p.k <= 12) return launch_router<L, NI, G, kFew>(p, loss, ctas, s);
    return launch_router<L, NI, G, NI>(p, loss, ctas, s);
}

// Calls f with the lanes of a token and the experts of a lane as template arguments.  Up to 64 experts 8 lanes have a
// token, so that a warp works on four (32767 tokens of 64 experts: 11.7 us, with 32 lanes 14.1; of 32: 7.4 and 13.1).
template <class F>
cudaError_t by_experts(int E, F f) {
    if (E <= 8) return f.template run<1, 8>();
    if (E <= 16) return f.template run<2, 8>();
    if (E <= 32) return f.template run<4, 8>();
    if (E <= 64) return f.template run<8, 8>();
    if (E <= 128) return f.template run<4, 32>();
    if (E <= 256) return f.template run<8, 32>();
    if (E <= 512) return f.template run<16, 32>();
    return f.template run<32, 32>();
}

struct RunRouter {
    const RouterParams &p;
    bool bf, loss, given;
    int ctas;
    cudaStream_t s;
    template <int NI, int G>
    cudaError_t run() const {
        return bf ? launch_router<bf16, NI, G>(p, loss, given, ctas, s) : launch_router<float, NI, G>(p, loss, given, ctas, s);
    }
};

struct RunBwd {
    const RouterBwd &p;
    bool bf;
    int ctas;
    cudaStream_t s;
    template <int NI, int G>
    cudaError_t run() const {
        const size_t smem = p.d_weights ? (size_t)kWarps * (32 / G) * p.E * 4 : 0;   // at most 32 KB
        if (bf) return launch(router_bwd_kernel<bf16, NI, G>, ctas, kThreads, smem, 1, s, p);
        return launch(router_bwd_kernel<float, NI, G>, ctas, kThreads, smem, 1, s, p);
    }
};

bool loss_ok(const moe_balance_io *l, const void *ws) {
    return l->num_seqs >= 1 && l->num_seqs <= MOE_MAX_SEQS && (l->seq_offsets || l->num_seqs == 1) && l->loss && l->counts && l->prob_mean &&
           l->seq_tokens && ws && aligned_to(ws, 256) && aligned_to(l->seq_offsets, 4) && aligned_to(l->loss, 4) &&
           aligned_to(l->counts, 4) && aligned_to(l->prob_mean, 4) && aligned_to(l->seq_tokens, 4);
}

int route(const moe_router_config *cfg, int T, const void *logits, int64_t ld, const float *bias, int32_t *idx,
          float *weights, bool given, const moe_balance_io *loss, void *ws, cudaStream_t s) {
    RouterParams p{};
    p.logits = logits;
    p.ld = ld;
    p.bias = bias;
    p.topk_idx = idx;
    p.topk_weights = weights;
    p.T = T;
    p.E = cfg->num_experts;
    p.k = cfg->topk;
    p.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
    p.renorm = cfg->renormalize != 0;
    p.score_bias = bias && cfg->bias_on == MOE_BIAS_SCORE;
    p.scale = cfg->weight_scale;
    p.S = loss ? loss->num_seqs : 1;
    p.seq_offsets = loss ? loss->seq_offsets : nullptr;
    const int ctas = ctas_for(T, p.E, p.S);
    p.chunk = T > 0 ? (T - 1) / ctas + 1 : 1;
    if (loss) carve(p.E, T, p.S, static_cast<char *>(ws), &p.part);
    if (T > 0) {
        if (by_experts(p.E, RunRouter{p, cfg->logits_dtype == MOE_DTYPE_BF16, loss != nullptr, given,
                                      (T - 1) / p.chunk + 1, s}) != cudaSuccess)
            return MOE_ERR_CUDA;
    } else if (loss && cudaMemsetAsync(p.part.ticket, 0, sizeof(int), s) != cudaSuccess) {
        return MOE_ERR_CUDA;
    }
    if (loss) {
        SumParams q{p.part, p.seq_offsets, loss->counts, loss->prob_mean, loss->seq_tokens, loss->loss, T, p.E, p.k, p.S,
                    p.chunk, cfg->balance_coef, cfg->z_coef};
        // 32 warps where a sequence has more rows than 8 can take in two turns (40397 tokens of 59 experts in one
        // sequence, losses and gradient: 47.8 us, with 8 warps 61.5)
        const unsigned sums = (unsigned)((p.E + 31) / 32) * p.S;
        const cudaError_t e = ctas > 16 * p.S ? launch(router_seq_kernel<32>, sums, 1024, 0, 1, s, q)
                                              : launch(router_seq_kernel<8>, sums, 256, 0, 1, s, q);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_workspace_bytes(const moe_router_config *cfg, int max_tokens, int max_seqs) {
    if (!valid(cfg) || max_tokens < 0 || max_seqs < 1 || max_seqs > MOE_MAX_SEQS) return 0;
    return carve(cfg->num_experts, max_tokens, max_seqs, nullptr, nullptr);
}

int moe_router_forward(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                       const float *bias, int32_t *topk_idx, float *topk_weights, const moe_balance_io *loss,
                       void *d_workspace, void *stream) {
    if (!valid(cfg) || num_tokens < 0 || (loss && !loss_ok(loss, d_workspace))) return MOE_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!logits || !topk_idx || !topk_weights || ld_logits < cfg->num_experts))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, dtype_bytes(cfg->logits_dtype)) || !aligned_to(bias, 4) || !aligned_to(topk_idx, 4) ||
        !aligned_to(topk_weights, 4))
        return MOE_ERR_INVALID_ARG;
    return route(cfg, num_tokens, logits, ld_logits, bias, topk_idx, topk_weights, false, loss, d_workspace,
                 static_cast<cudaStream_t>(stream));
}

int moe_balance_loss(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                     const int32_t *topk_idx, const moe_balance_io *loss, void *d_workspace, void *stream) {
    if (!valid(cfg) || num_tokens < 0 || !loss || !loss_ok(loss, d_workspace)) return MOE_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!logits || !topk_idx || ld_logits < cfg->num_experts)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, dtype_bytes(cfg->logits_dtype)) || !aligned_to(topk_idx, 4)) return MOE_ERR_INVALID_ARG;
    return route(cfg, num_tokens, logits, ld_logits, nullptr, const_cast<int32_t *>(topk_idx), nullptr, true, loss,
                 d_workspace, static_cast<cudaStream_t>(stream));
}

int moe_router_backward(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                        const int32_t *topk_idx, const float *d_weights, const moe_balance_io *loss,
                        const float *d_loss, void *d_logits, int64_t ld_d_logits, void *stream) {
    if (!valid(cfg) || num_tokens < 0 || (!d_weights && !d_loss)) return MOE_ERR_INVALID_ARG;
    if (d_loss && (!loss || loss->num_seqs < 1 || loss->num_seqs > MOE_MAX_SEQS || (!loss->seq_offsets && loss->num_seqs != 1) ||
                   !loss->counts || !loss->seq_tokens || !aligned_to(loss->seq_offsets, 4) || !aligned_to(loss->counts, 4) ||
                   !aligned_to(loss->seq_tokens, 4)))
        return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    const size_t es = dtype_bytes(cfg->logits_dtype);
    if (!logits || !d_logits || (d_weights && !topk_idx) || ld_logits < cfg->num_experts ||
        ld_d_logits < cfg->num_experts)
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(d_logits, es) || !aligned_to(topk_idx, 4) || !aligned_to(d_weights, 4) ||
        !aligned_to(d_loss, 4))
        return MOE_ERR_INVALID_ARG;
    RouterBwd p{};
    p.logits = logits;
    p.ld = ld_logits;
    p.topk_idx = topk_idx;
    p.d_weights = d_weights;
    if (d_loss) {
        p.seq_offsets = loss->seq_offsets;
        p.counts = loss->counts;
        p.seq_tokens = loss->seq_tokens;
        p.S = loss->num_seqs;
    }
    p.d_loss = d_loss;
    p.d_logits = d_logits;
    p.ld_d = ld_d_logits;
    p.T = num_tokens;
    p.E = cfg->num_experts;
    p.k = cfg->topk;
    p.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
    p.renorm = cfg->renormalize != 0;
    p.scale = cfg->weight_scale;
    p.alpha = cfg->balance_coef;
    p.beta = cfg->z_coef;
    const int ctas = ctas_for(num_tokens, p.E, p.S);
    p.chunk = (num_tokens - 1) / ctas + 1;
    return by_experts(p.E, RunBwd{p, cfg->logits_dtype == MOE_DTYPE_BF16, (num_tokens - 1) / p.chunk + 1,
                                  static_cast<cudaStream_t>(stream)}) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // extern "C"
