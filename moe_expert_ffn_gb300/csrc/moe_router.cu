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
#include "moe_router.cuh"

namespace moe {
namespace {

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
    const Experts<NI, G, false> x(RouterParams{}, lg);
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
            load_row(raw, p.logits, p.ld, tw + grp, tw + grp < end, lg, E, x);
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
            if (tn < end) load_row(raw, p.logits, p.ld, tn + grp, tn + grp < end, lg, E, x);
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
    if (c->num_groups != 0) {
        if (c->num_groups < 2 || c->num_groups > 32 || c->num_experts % c->num_groups) return false;
        const int size = c->num_experts / c->num_groups;
        if (c->num_groups * ((size + 31) / 32) > 32) return false;
        if (c->topk_groups < 1 || c->topk_groups > c->num_groups || c->topk > c->topk_groups * size) return false;
        if (c->group_score != MOE_GROUP_MAX && c->group_score != MOE_GROUP_TOP2) return false;
    }
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
    // all groups: by logits the choice is that without groups; by scores it is not, whose keys without groups are approximate
    if (cfg->num_groups && !given && (cfg->topk_groups < cfg->num_groups || cfg->bias_on == MOE_BIAS_SCORE)) {
        p.groups = cfg->num_groups;
        p.group_size = p.E / p.groups;
        p.use_groups = cfg->topk_groups;
        p.top2 = cfg->group_score == MOE_GROUP_TOP2 && p.group_size > 1;
        const int by8 = (p.group_size + 7) / 8;
        p.each = p.groups * by8 <= 8 ? by8 : (p.group_size + 31) / 32;
        p.score_bias = cfg->bias_on == MOE_BIAS_SCORE;   // without a bias too: a group's sum is of scores
    }
    p.scale = cfg->weight_scale;
    p.S = loss ? loss->num_seqs : 1;
    p.seq_offsets = loss ? loss->seq_offsets : nullptr;
    const int held = p.groups * p.each;   // with groups, registers of a lane
    const int ctas = std::min(ctas_for(T, p.E, p.S), loss && held > 4 && held <= 8 ? kMaxCtas / 4 * ctas_an_sm(8, true) : kMaxCtas);
    p.chunk = T > 0 ? (T - 1) / ctas + 1 : 1;
    if (loss) carve(p.E, T, p.S, static_cast<char *>(ws), &p.part);
    if (T > 0 && p.groups > 1) {
        const auto run = cfg->logits_dtype == MOE_DTYPE_BF16 ? launch_router_groups_bf16 : launch_router_groups_f32;
        if (run(p, loss != nullptr, (T - 1) / p.chunk + 1, s) != cudaSuccess)
            return MOE_ERR_CUDA;
    } else if (T > 0) {
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
