// moe_router.cuh -- the router's forward kernel (choice, weights, partial sums of the losses), instantiated without groups in
// moe_router.cu and with them in moe_router_groups*.cu.
#pragma once

#include <float.h>
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {

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
    int groups, group_size, use_groups, top2;   // groups > 1: the choice is limited to the best use_groups groups
    int each;                                   // registers of a lane for a group
    float scale;
};

// moe_router_groups*.cu: a forward pass whose choice is limited to groups.
cudaError_t launch_router_groups_f32(const RouterParams &p, bool loss, int ctas, cudaStream_t s);
cudaError_t launch_router_groups_bf16(const RouterParams &p, bool loss, int ctas, cudaStream_t s);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 608;   // four on each of 152 SMs
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.44269504f;

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

// Which experts a lane holds: lg, lg + G, ...; with groups (kGrouped) a group takes `each` registers of every lane, so that a
// group's experts are in registers of their own: register i holds place lg + G (i % each) of group i / each.
template <int NI, int G, bool kGrouped>
struct Experts {
    int off[kGrouped ? NI : 1];
    uint32_t has_bits = 0;
    __device__ __forceinline__ Experts(const RouterParams &p, int lg) {
        if constexpr (kGrouped) {
#pragma unroll
            for (int i = 0, g = 0, j = 0; i < NI; ++i) {
                off[i] = g * p.group_size + j * G;
                if (g < p.groups && j * G + lg < p.group_size) has_bits |= 1u << i;
                if (++j == p.each) j = 0, ++g;
            }
        }
    }
    __device__ __forceinline__ int at(int i, int lg) const {
        if constexpr (kGrouped) return off[i] + lg;
        return lg + G * i;
    }
    __device__ __forceinline__ bool has(int i, int lg, int E) const {
        if constexpr (kGrouped) return (has_bits >> i) & 1;
        return lg + G * i < E;
    }
};

// A token's logits as loaded (-inf where there is none), so that the next token's can be on their way.
template <class L, int NI, int G, bool kGrouped = false>
__device__ __forceinline__ void load_row(L (&l)[NI], const void *logits, int64_t ld, uint32_t t, bool on, int lg, int E,
                                         const Experts<NI, G, kGrouped> &x) {
    const L *row = static_cast<const L *>(logits) + (int64_t)t * ld + lg;
    if (E == NI * G) {   // every lane has all its experts
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = on ? row[G * i] : from_f32<L>(-INFINITY);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = on && x.has(i, lg, E) ? row[x.at(i, 0)] : from_f32<L>(-INFINITY);
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

// The k largest keys of a group's token from the full keys, one by one: the exact choice whatever the keys.  Returns whether
// two neighbours among them, or the last one and the first left out, are no further apart than `margin` (of use where it is
// not negative).
template <int NI, int G, int NS>
__device__ __noinline__ bool choose_exact(const float (&key)[NI], int k, int lg, float margin, int (&slot_e)[NS]) {
    uint32_t taken = 0;
    bool close = false;
    float above = INFINITY;
    const int rounds = margin >= 0.0f ? k + 1 : k;
#pragma unroll
    for (int q = 0; q < NS; ++q) slot_e[q] = -1;
    for (int j = 0; j < rounds; ++j) {
        float best = -INFINITY;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (!((taken >> i) & 1) && key[i] > best) best = key[i], bi = i;   // of equal keys the first stays
        const float m = group_max<G>(best);
        close |= above - m <= margin;   // -inf: nothing is left, no neighbour
        above = m > -INFINITY ? m : INFINITY;
        int e = group_min<G>(best == m && m > -INFINITY ? lg + G * bi : 1 << 20);
        if (e < 1 << 20) {
            if ((e & (G - 1)) == lg) taken |= 1u << (e / G);
        } else {
            e = -1;
        }
#pragma unroll
        for (int q = 0; q < NS; ++q)
            if (j == q * G + lg && j < k) slot_e[q] = e;
    }
    return close;
}

// A float as a whole number of the same order, and back.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are equal
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}

// The k largest keys of a group's token, ties to the lowest expert.  Slot j goes to lane j % G, place j / G: its expert
// (-1: nothing left).  `exact`: the keys' low bits that the expert's number takes say nothing.  A lane keeps its D
// largest; one that wins D < NI times may have had more.  Returns false, with nothing chosen, where a key is +inf or a
// NaN that sorts above it and `cleaned` does not say that it is meant.  kMargin: keys are right within margin / 2 (their order is
// known where they are further apart than that); chosen ones that are not are ranked by exact_of, and `close` says whether
// candidates for the last place are left that are not.
template <int NI, int G, int NS, int D, bool kMargin = false, class Exact = int>
__device__ __forceinline__ bool choose(const float (&key)[NI], int k, int lg, bool exact, bool cleaned, int (&slot_e)[NS],
                                       float margin = -1.0f, bool *close = nullptr, Exact exact_of = Exact()) {
    constexpr uint32_t kLow = (uint32_t)(NI * G - 1);   // bits of an expert's number
    constexpr uint32_t kOpen = 0x00800000u;             // the order of the smallest finite float
    auto packed = [&](int i) { return (ordered(key[i]) & ~kLow) | (kLow - (uint32_t)(lg + G * i)); };
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
        uint32_t least = max(exact ? last : last & ~kLow, kOpen);
        if (kMargin) least = max(ordered(from_ordered(least) - margin) & ~kLow, kOpen);
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
            if (kMargin) {   // by the high bits and the margin together
                const float hi = from_ordered(slot[q] & ~kLow), lo = from_ordered(next | kLow);
                const bool same = q * G + lg < k && slot[q] >= kOpen && next >= kOpen && hi - lo <= margin;
                near |= same && !edge;
                again |= same && (edge || NS > 1);
                continue;
            }
            const bool same = q * G + lg < k && slot[q] >= kOpen && ((slot[q] ^ next) & ~kLow) == 0;
            near |= same && !edge;
            again |= same && (edge || NS > 1);
        }
        if constexpr (kMargin && NS == 1) {
            again |= near && k > G - 2;
            const bool set = __any_sync(kAll, again);
            if (k <= G - 2 && (set || __any_sync(kAll, near))) {
                // ranked anew by exact keys; where it is the last place that is not sure, the first k + 2 by the keys at hand, of
                // which the last has to end more than the margin below the k-th, lest others belong among them
                int place[1] = {lg < k ? slot_e[0] : -1};
                if (set) choose_exact<NI, G, 1>(key, k + 2, lg, -1.0f, place);
                const int m = set ? k + 2 : k, at = place[0];
                const float mine = at >= 0 ? exact_of(at) : -INFINITY;
                int rank = 0;   // empty slots stay behind all others
#pragma unroll 1
                for (int j = 0; j < m; ++j) {
                    const float f = __shfl_sync(kAll, mine, j, G);
                    const int fe = __shfl_sync(kAll, at, j, G);
                    rank += f > mine || (f == mine && fe >= 0 && fe < at);
                }
                if (lg >= m || at < 0) rank = G;
                const float least = group_max<G>(rank >= k - 1 ? mine : -INFINITY), last = __shfl_sync(kAll, mine, k + 1, G);
                *close = set && last > -INFINITY && least - last <= margin;
                slot_e[0] = -1;
#pragma unroll 1
                for (int j = 0; j < m; ++j) {
                    const int r = __shfl_sync(kAll, rank, j, G), fe = __shfl_sync(kAll, at, j, G);
                    if (r == lg && lg < k) slot_e[0] = fe;
                }
                return true;
            }
        } else if (NS == 1 && __any_sync(kAll, near) && !__any_sync(kAll, again)) {
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
    if (!__any_sync(kAll, again)) return true;
    const bool c = choose_exact<NI, G, NS>(key, k, lg, kMargin ? margin : -1.0f, slot_e);
    if (kMargin) *close = c;
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
// six 20.6 to 22; 28219 x 259: two 20.4, one 29.2).  With both groups and losses (`both`) three: 32768 x 256 bf16 in 4 groups,
// losses and gradient 51 us, with four 58; of scores in 8 groups 77, with four and the scores by a call 83.
constexpr int ctas_an_sm(int NI, bool both = false) { return NI == 8 && both ? 3 : NI <= 8 ? 4 : NI == 16 ? 2 : 1; }

// A group's score from what its lanes hold of it, their largest key and (top2) their second.
template <int G>
__device__ __forceinline__ float group_score(float first, float second, bool top2) {
    float s = group_max<G>(first);
    if (top2) {
        const unsigned best = __ballot_sync(kAll, first == s) >> (threadIdx.x & 31 & ~(G - 1)) & (G == 32 ? kAll : (1u << G) - 1);
        float t = group_max<G>(first == s ? second : first);
        if (best & (best - 1)) t = s;
        s += t > -INFINITY ? t : 0.0f;
    }
    return s;
}

// Closes the experts outside the best use_groups groups of a token: a group's score is its largest key, or the sum of its two
// largest (of one open expert's, that alone), ties go to the lowest group.  Returns whether the scores of the last group taken
// and the best one left out are within `margin`.  kEach: registers that a group is of every lane, 0 where p.each says.
template <int NI, int G, int kEach>
__device__ __forceinline__ bool keep_groups(float (&key)[NI], const RouterParams &p, int lg, float margin) {
    float score = -INFINITY;   // of group lg, groups <= G
    if (kEach) {
#pragma unroll
        for (int g = 0; g < NI / (kEach ? kEach : 1); ++g) {
            float first = key[g * kEach], second = -INFINITY;
#pragma unroll
            for (int j = 1; j < kEach; ++j) {
                const float v = key[g * kEach + j];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
            const float s = group_score<G>(first, second, p.top2);
            if (lg == g) score = s;
        }
    } else {
        float first = -INFINITY, second = -INFINITY;
#pragma unroll
        for (int i = 0, g = 0, j = 0; i < NI; ++i) {
            second = fmaxf(second, fminf(first, key[i]));
            first = fmaxf(first, key[i]);
            if (++j == p.each) {
                const float s = group_score<G>(first, second, p.top2);
                if (lg == g) score = s;
                first = second = -INFINITY;
                j = 0, ++g;
            }
        }
    }
    int rank = 0;
    if (kEach == 1 && G == 32 && NI == 8) {
        // four lanes to a group, each comparing it with two others
        const int g = lg & 7;
        const float own = __shfl_sync(kAll, score, g);
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
            const int h = (lg >> 3) + q;
            const float s = __shfl_sync(kAll, score, h);
            rank += __popc(__ballot_sync(kAll, s > own || (s == own && h < g)) & (0x01010101u << g));
        }
    } else if (kEach) {   // groups that are not there have no better score
#pragma unroll
        for (int g = 0; g < NI / (kEach ? kEach : 1); ++g) {
            const float s = __shfl_sync(kAll, score, g, G);
            rank += s > score || (s == score && g < lg);
        }
    } else {
#pragma unroll 8
        for (int g = 0; g < p.groups; ++g) {
            const float s = __shfl_sync(kAll, score, g, G);
            rank += s > score || (s == score && g < lg);
        }
    }
    const bool taken = rank < p.use_groups && lg < p.groups;
    const unsigned mask = __ballot_sync(kAll, taken) >> (threadIdx.x & 31 & ~(G - 1));
#pragma unroll
    for (int i = 0, g = 0, j = 0; i < NI; ++i) {
        if (!((mask >> (kEach ? i / (kEach ? kEach : 1) : g)) & 1)) key[i] = -INFINITY;
        if (!kEach && ++j == p.each) j = 0, ++g;
    }
    if (margin < 0.0f) return false;
    const float left = group_max<G>(taken ? -INFINITY : score);
    return __any_sync(kAll, taken && score > -INFINITY && score - left <= margin);
}

// The same for the few tokens that need it twice, in little code: code that is seldom run is fetched when it is (one such token
// among 128 took 2.4 us).
template <int NI, int G>
__device__ __noinline__ void keep_groups_again(float (&key)[NI], const RouterParams &p, int lg) {
    float score = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
        float first = -INFINITY, second = -INFINITY;
#pragma unroll 1
        for (int i = g * p.each; i < (g + 1) * p.each; ++i) {
            second = fmaxf(second, fminf(first, key[i]));
            first = fmaxf(first, key[i]);
        }
        const float s = group_score<G>(first, second, p.top2);
        if (lg == g) score = s;
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
        const float s = __shfl_sync(kAll, score, g, G);
        rank += s > score || (s == score && g < lg);
    }
    const unsigned mask = __ballot_sync(kAll, rank < p.use_groups && lg < p.groups) >> (threadIdx.x & 31 & ~(G - 1));
#pragma unroll 1
    for (int i = 0; i < p.groups * p.each; ++i)
        if (!((mask >> (i / p.each)) & 1)) key[i] = -INFINITY;
}

// sigmoid(l) as a pair of floats within 2^-44 of itself, and rounded once: the order of scores that f32 arithmetic leaves open (sums and
// products with their exact errors by the methods of Dekker and Knuth; in 64 bits, whose units are few, a token that needs them held
// up the rest: 32767 x 256 44 us, in pairs 40).  With y = |l| - n ln 2 (ln 2 in parts, the first short enough for n times it to be
// exact, by Cody and Waite), e^-|l| is 2^-n times e^-y, and that the 256th power of e^(-y / 256), by its series; powers by w -> 2 w +
// w^2 on what they are above 1.  (The 64th power of e^(-y / 64) is within 2^-40.6: the series' last terms, rounded, 64 times.)
__device__ __noinline__ float score_exact(float l) {
    if (!(l > -INFINITY)) return -INFINITY;
    if (l >= 32.0f) return 1.0f;
    const float a = fminf(fabsf(l), 110.0f), n = rintf(a * kLog2e);
    constexpr float kLn2Mid = 2.12194440e-4f;   // ln 2 = 0.693359375 - (mid + low)
    constexpr float kLn2Low = (float)(0.693359375 - 0.69314718055994530942 - (double)kLn2Mid);
    const float r = fmaf(-n, 0.693359375f, a), p = __fmul_rn(n, kLn2Mid), e = fmaf(n, kLn2Low, fmaf(n, kLn2Mid, -p));
    const float yh = r + p, z = yh - r, yl = (r - (yh - z)) + (p - z) + e;
    const float xh = yh * -0x1p-8f, xl = yl * -0x1p-8f, sq = __fmul_rn(xh, xh), sl = fmaf(xh, xh, -sq) + 2.0f * xh * xl;
    const float tail = sq * xh * fmaf(xh, fmaf(xh, fmaf(xh, 1.0f / 720, 1.0f / 120), 1.0f / 24), 1.0f / 6);
    float wh = xh + 0.5f * sq, wl = (xh - wh) + 0.5f * sq + (xl + 0.5f * sl + tail);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const float ph = __fmul_rn(wh, wh), pl = fmaf(wh, wh, -ph) + 2.0f * wh * wl;
        const float h = 2.0f * wh + ph, low = (2.0f * wh - h) + ph + (2.0f * wl + pl);
        wh = h + low;
        wl = (h - wh) + low;
    }
    const float gh = 1.0f + wh, gl = (1.0f - gh) + wh + wl, down = n > 126.0f ? 0.0f : ldexpf(1.0f, -(int)n);
    const float th = gh * down, tl = gl * down, dh = 1.0f + th, dl = (1.0f - dh) + th + tl;
    const float q = __frcp_rn(dh), ql = q * fmaf(-q, dl, fmaf(-q, dh, 1.0f));   // 1 / (1 + e^-|l|)
    if (l >= 0.0f) return q + ql;
    const float ph = __fmul_rn(gh, q), pl = fmaf(gh, q, -ph) + (gh * ql + gl * q);
    if (n < 126.0f) return ldexpf(ph + pl, -(int)n);
    // below the normal numbers, or next to them: in units of 2^-149 from 46 bits behind the point, so that it is rounded once
    const int drop = (int)n - 103;
    const long long v = (long long)(ph * 0x1p46f) + (long long)(pl * 0x1p46f);
    return __int_as_float((int)((v + (1ll << (drop - 1))) >> drop));
}

// How far apart two keys (scores plus bias), or two sums of two keys, must be for their f32 order to be that of the exact ones:
// a score is within 2^-21 of the exact one (score_of: its exponential within 2^-22 + 1.7 |l| 2^-24 of itself, the quotient within
// 2^-22; either error shrinks with the score), so the difference of two sums is within 2^-19; and each of the up to six sums
// that enter it, approximate and exact, rounds to 2^-24 of the largest key or twice that: under 2^-20 of it in all.  `bias`: the
// largest finite one's magnitude, which with a score of 1 bounds every key that is not infinite.
__device__ __forceinline__ float score_margin(float bias) { return fmaf(1.0f + bias, 0x1p-20f, 0x1p-19f); }

// The choice limited to groups.
template <class L, int NI, int G, int NS, int D, int kEach>
__device__ __forceinline__ void choose_grouped(float (&l)[NI], const float (&bias)[NI], float margin, const RouterParams &p, uint32_t t, int lg,
                                               bool exact, int (&slot_e)[NS]) {
    auto expert_of = [&](int place) { return p.E == NI * G ? place : place / (p.each * G) * p.group_size + place % (p.each * G); };
    auto exact_of = [&](int place) {
        const int e = expert_of(place);
        const float l1 = open_logit(to_f32(static_cast<const L *>(p.logits)[(int64_t)t * p.ld + e]));
        const float s = score_exact(l1);
        return p.bias ? s + p.bias[e] : s;
    };
    float key[NI];
    bool close = false, edge = false;
    // a score of a NaN is closed, of +inf 1, as of the largest logit
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        key[i] = p.score_bias ? score_of(l[i]) : open_logit(l[i]);
        if (p.bias) key[i] = fmaxf(key[i] + bias[i], -INFINITY);
    }
    if (p.score_bias) {
        close = keep_groups<NI, G, kEach>(key, p, lg, margin);
        choose<NI, G, NS, D, true>(key, p.k, lg, false, true, slot_e, margin, &edge, exact_of);
    } else {
        keep_groups<NI, G, kEach>(key, p, lg, -1.0f);
        choose<NI, G, NS, D>(key, p.k, lg, exact, true, slot_e);
    }
    if (__any_sync(kAll, close || edge)) {
        // two scores that decide the groups, or several candidates for the last place: once more by exact ones
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            key[i] = score_exact(open_logit(l[i]));
            if (p.bias) key[i] = fmaxf(key[i] + bias[i], -INFINITY);
        }
        keep_groups_again<NI, G>(key, p, lg);
        choose_exact<NI, G, NS>(key, p.k, lg, -1.0f, slot_e);
    }
#pragma unroll
    for (int q = 0; q < NS; ++q)
        if (slot_e[q] >= 0) slot_e[q] = expert_of(slot_e[q]);
}

// kGrouped: 0, or with groups of any size 1, of one register a lane 2, of two 3 (32768 x 256 bf16 in 4 groups, losses and gradient
// 64 us by the form for any size, 58).
template <class L, int NI, int G, int D, bool kLoss, bool kGiven, int kGrouped = 0>
__global__ void __launch_bounds__(kThreads, ctas_an_sm(NI, kGrouped && kLoss)) router_kernel(const __grid_constant__ RouterParams p) {
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
    const Experts<NI, G, kGrouped != 0> x(p, lg);
    float bias[NI];
    if (!kGiven && p.bias) {
#pragma unroll
        for (int i = 0; i < NI; ++i) bias[i] = x.has(i, lg, E) ? p.bias[x.at(i, lg)] : 0.0f;
    }
    float margin = 0.0f;
    if (kGrouped) {
        if (p.score_bias && p.bias) {
#pragma unroll
            for (int i = 0; i < NI; ++i) margin = fmaxf(margin, fabsf(bias[i]) < INFINITY ? fabsf(bias[i]) : 0.0f);
            margin = group_max<G>(margin);
        }
        margin = score_margin(margin);
    }
    int s_at = 0;
    for (int a = t0; a < t1;) {
        const Cut cut = kLoss ? cut_at(p.seq_offsets, p.S, a, t1, s_at) : Cut{0, t1, true};
        s_at = cut.s;
        L raw[NI];
        const uint32_t end = cut.end, tw = (uint32_t)a + warp * kGroups;   // a step past the last token may pass 2^31
        if (tw < end) load_row(raw, p.logits, p.ld, tw + grp, tw + grp < end, lg, E, x);
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
            if (tn < end) load_row(raw, p.logits, p.ld, tn + grp, tn + grp < end, lg, E, x);
            float m = -INFINITY, top = -INFINITY;   // the largest logit, and that of the chosen
            if (kGiven || (kLoss && (p.bias || kGrouped)) || (!p.renorm && !p.sigmoid)) {
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
                if constexpr (kGrouped) {
                    choose_grouped<L, NI, G, NS, D, kGrouped - 1>(l, bias, margin, p, t, lg, sizeof(L) == 2 && !p.bias && !p.score_bias, my_e);
                } else for (int pass = 0; pass < 2; ++pass) {
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
                    if (kLoss && !kGrouped && !p.bias) m = top;
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
                const float pr = over_groups<G>(prob[i]);
                if (x.has(i, lg, E) && grp == 0) joined[warp * E + x.at(i, lg)] = pr;
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

}  // namespace
}  // namespace moe
