// moe_router.cu -- the top-k router, the balance and z losses with per-sequence
// expert counts, and the gradient of the logits (definitions in
// include/moe.h).
//
// One warp per token; lane l holds experts l, l + 32, ...  Every warp walks a
// contiguous range of tokens and keeps its loss sums in registers until the
// sequence changes; then it writes them to a row of partial sums of its own.
// Warp w in sequence s uses row w + s: along the walk either one grows with
// every new pair, so rows never collide, and the rows of a sequence are those
// of the consecutive warps that its tokens fall on.  The sums over rows are
// taken in row order: no atomics, the same bits every time.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "moe.h"
#include "moe_device.cuh"
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kMaxLossWarps = 2432;   // 16 warps on each of 152 SMs
constexpr unsigned kAll = 0xFFFFFFFFu;

// Rows of partial sums and what follows them in the workspace.
struct Partials {
    float *prob;     // [rows][E]
    int32_t *count;  // [rows][E]
    float *z;        // [rows]
    int32_t *tokens; // [rows]
    float *seq_bal;  // [S]
    float *seq_z;    // [S]
};

struct RouterParams {
    const void *logits;
    int64_t ld;
    const float *bias;
    int32_t *topk_idx;          // out, or in with kGiven
    float *topk_weights;
    const int32_t *seq_offsets;
    Partials part;
    int T, E, k, S, chunk;      // chunk: tokens per warp
    int sigmoid, renorm;
    float scale;
};

// Keys whose order as unsigned integers is the order of the floats; 0 for a
// closed expert (-inf or NaN).
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are equal
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// A logit as it enters the scores: closed ones -inf, +inf the largest float.
__device__ __forceinline__ float open_logit(float v) { return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY; }

// Sigmoid times e^-m with m = min(largest logit, 0): the ratios of the scores
// of a token whose sigmoids all underflow stay right.
__device__ __forceinline__ float sigmoid_scaled(float l, float m) {
    return l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / (1.0f + expf(l));
}

__device__ __forceinline__ int find_seq(const int32_t *off, int S, int t) {
    int lo = 0, hi = S;   // first s with off[s + 1] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

template <class L, int NI, bool kLoss, bool kGiven>
__global__ void __launch_bounds__(kThreads) router_kernel(const RouterParams p) {
    const int lane = threadIdx.x & 31;
    const int w = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    const int t0 = (int)min((int64_t)w * p.chunk, (int64_t)p.T), t1 = min(t0 + p.chunk, p.T);
    if (t0 >= t1) return;
    float prob[kLoss ? NI : 1];
    int cnt[kLoss ? NI : 1];
    float zsum = 0.0f;
    int tokens = 0, s = 0, s_begin = 0, s_end = p.T;
    if (kLoss) {
#pragma unroll
        for (int i = 0; i < NI; ++i) prob[i] = 0.0f, cnt[i] = 0;
        if (p.seq_offsets) {
            s = find_seq(p.seq_offsets, p.S, t0);
            s_begin = s < p.S ? p.seq_offsets[s] : p.T;
            s_end = s < p.S ? p.seq_offsets[s + 1] : p.T;
        }
    }
    auto flush = [&]() {
        const int64_t row = (int64_t)w + s;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E) {
                p.part.prob[row * p.E + e] = prob[i];
                p.part.count[row * p.E + e] = cnt[i];
            }
            prob[i] = 0.0f;
            cnt[i] = 0;
        }
        if (lane == 0) {
            p.part.z[row] = zsum;
            p.part.tokens[row] = tokens;
        }
        zsum = 0.0f;
        tokens = 0;
    };
    for (int t = t0; t < t1; ++t) {
        if (kLoss && p.seq_offsets && t >= s_end) {
            flush();
            s = find_seq(p.seq_offsets, p.S, t);
            s_begin = s < p.S ? p.seq_offsets[s] : p.T;
            s_end = s < p.S ? p.seq_offsets[s + 1] : p.T;
        }
        const L *row = static_cast<const L *>(p.logits) + t * p.ld;
        float l[NI];
        uint32_t key[NI];
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 32 * i;
            l[i] = open_logit(e < p.E ? to_f32(row[e]) : -INFINITY);
            m = fmaxf(m, l[i]);
            if (!kGiven) key[i] = e < p.E ? order_key(p.bias ? l[i] + p.bias[e] : l[i]) : 0u;
            if (!kGiven && !(l[i] > -INFINITY)) key[i] = 0u;
        }
        m = warp_max(m);
        uint32_t mask = 0;   // bit i: expert lane + 32 i is chosen
        if (kGiven) {
            const int idx = lane < p.k ? p.topk_idx[(int64_t)t * p.k + lane] : -1;
            for (int j = 0; j < p.k; ++j) {
                const int e = __shfl_sync(kAll, idx, j);
                if (e >= 0 && e < p.E && (e & 31) == lane) mask |= 1u << (e >> 5);
            }
        } else {
            int my_e = -1;          // lane j: slot j
            float my_l = -INFINITY;
            for (int j = 0; j < p.k; ++j) {
                uint32_t best = 0;
#pragma unroll
                for (int i = 0; i < NI; ++i) best = max(best, key[i]);
                const uint32_t top = __reduce_max_sync(kAll, best);
                if (top == 0) break;
                int e = 1 << 20;
                float v = 0.0f;
#pragma unroll
                for (int i = NI - 1; i >= 0; --i)
                    if (key[i] == top) e = lane + 32 * i, v = l[i];
                const int win = __reduce_min_sync(kAll, (unsigned)e);
                v = __shfl_sync(kAll, v, win & 31);
                if (e == win) {
                    mask |= 1u << (win >> 5);
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        if (i == (win >> 5)) key[i] = 0u;
                }
                if (lane == j) my_e = win, my_l = v;
            }
            // weights of the chosen
            float wgt = 0.0f;
            if (p.renorm || p.sigmoid) {
                const float top_l = warp_max(my_l);
                if (my_e >= 0)
                    wgt = !p.sigmoid ? expf(my_l - top_l) : sigmoid_scaled(my_l, p.renorm ? fminf(top_l, 0.0f) : 0.0f);
                if (p.renorm) {
                    const float sum = warp_sum(wgt);
                    wgt = sum > 0.0f ? wgt / sum : 0.0f;
                }
            } else {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) z += l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
                z = warp_sum(z);
                if (my_e >= 0) wgt = expf(my_l - m) / z;
            }
            if (lane < p.k) {
                p.topk_idx[(int64_t)t * p.k + lane] = my_e;
                p.topk_weights[(int64_t)t * p.k + lane] = wgt * p.scale;
            }
        }
        if (kLoss && m > -INFINITY && t >= s_begin && t < s_end) {
            float q[NI], z = 0.0f;
            const float ms = fminf(m, 0.0f);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                q[i] = !(l[i] > -INFINITY) ? 0.0f : p.sigmoid ? sigmoid_scaled(l[i], ms) : expf(l[i] - m);
                z += q[i];
            }
            z = warp_sum(z);
            const float inv = 1.0f / z;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                prob[i] += q[i] * inv;
                cnt[i] += (mask >> i) & 1;
            }
            const float lse = m + logf(z);
            zsum += p.sigmoid ? 0.0f : lse * lse;
            ++tokens;
        }
    }
    if (kLoss) flush();
}

struct SumParams {
    Partials part;
    const int32_t *seq_offsets;
    int32_t *counts;
    float *prob_mean;
    int32_t *seq_tokens;
    int T, E, k, S, chunk;
};

// One CTA per sequence: its rows summed in order, then its share of the losses.
__global__ void __launch_bounds__(kThreads) router_seq_kernel(const SumParams p) {
    __shared__ float red[kWarpsPerCta];
    const int s = blockIdx.x;
    const int a = p.seq_offsets ? max(0, min(p.seq_offsets[s], p.T)) : 0;
    const int b = p.seq_offsets ? max(0, min(p.seq_offsets[s + 1], p.T)) : p.T;
    const int w0 = a / p.chunk, w1 = b > a ? (b - 1) / p.chunk + 1 : w0;
    int n = 0;
    float z = 0.0f;
    for (int w = w0; w < w1; ++w) {
        n += p.part.tokens[w + s];
        z += p.part.z[w + s];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    float bal = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        float ps = 0.0f;
        int c = 0;
        for (int w = w0; w < w1; ++w) {
            ps += p.part.prob[(int64_t)(w + s) * p.E + e];
            c += p.part.count[(int64_t)(w + s) * p.E + e];
        }
        p.counts[(int64_t)s * p.E + e] = c;
        p.prob_mean[(int64_t)s * p.E + e] = ps * inv;
        bal += (float)c * (ps * inv);
    }
    bal = block_sum<kWarpsPerCta>(bal, red);
    if (threadIdx.x == 0) {
        p.seq_tokens[s] = n;
        p.part.seq_bal[s] = bal * ((float)p.E / (float)p.k) * inv;
        p.part.seq_z[s] = z;
    }
}

__global__ void router_loss_kernel(const Partials part, int S, int32_t *seq_tokens, float alpha, float beta, float *loss) {
    // one warp, sequences in a fixed order
    const int lane = threadIdx.x;
    float bal = 0.0f, z = 0.0f;
    int used = 0, n = 0;
    for (int s = lane; s < S; s += 32) {
        bal += part.seq_bal[s];
        z += part.seq_z[s];
        used += seq_tokens[s] > 0;
        n += seq_tokens[s];
    }
    bal = warp_sum(bal);
    z = warp_sum(z);
    used = __reduce_add_sync(kAll, used);
    n = __reduce_add_sync(kAll, n);
    if (lane == 0) {
        bal = used > 0 ? alpha * bal / (float)used : 0.0f;
        z = n > 0 ? beta * z / (float)n : 0.0f;
        loss[0] = bal + z;
        loss[1] = bal;
        loss[2] = z;
        seq_tokens[S] = used;
        seq_tokens[S + 1] = n;
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
    int T, E, k, S, sigmoid, renorm;
    float scale, alpha, beta;
};

template <class L, int NI>
__global__ void __launch_bounds__(kThreads) router_bwd_kernel(const RouterBwd p) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const L *row = static_cast<const L *>(p.logits) + (int64_t)t * p.ld;
    float l[NI], q[NI], d[NI], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        l[i] = open_logit(e < p.E ? to_f32(row[e]) : -INFINITY);
        m = fmaxf(m, l[i]);
        d[i] = 0.0f;
    }
    m = warp_max(m);
    const bool real = m > -INFINITY;
    const float ms = fminf(m, 0.0f);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        q[i] = !(l[i] > -INFINITY) ? 0.0f : p.sigmoid ? sigmoid_scaled(l[i], ms) : expf(l[i] - m);
        z += q[i];
    }
    z = warp_sum(z);
    const float inv = real ? 1.0f / z : 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) q[i] *= inv;
    if (p.d_loss && real) {
        int s = 0;
        bool inside = true;
        if (p.seq_offsets) {
            s = find_seq(p.seq_offsets, p.S, t);
            inside = s < p.S && t >= p.seq_offsets[s];
        }
        const int n = inside ? p.seq_tokens[s] : 0;
        if (n > 0) {
            const float g = *p.d_loss;
            const float c0 = g * p.alpha * (float)p.E / ((float)p.k * (float)n * (float)n * (float)p.seq_tokens[p.S]);
            const float zc = p.sigmoid ? 0.0f : g * 2.0f * p.beta / (float)p.seq_tokens[p.S + 1] * (m + logf(z));
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = lane + 32 * i;
                d[i] = e < p.E ? c0 * (float)p.counts[(int64_t)s * p.E + e] : 0.0f;
                dot += d[i] * q[i];
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                d[i] = q[i] * (d[i] - dot + zc);
                if (p.sigmoid && l[i] > -INFINITY) d[i] /= 1.0f + expf(l[i]);   // ds/dl = s (1 - s)
            }
        }
    }
    if (p.d_weights) {
        int idx = lane < p.k ? p.topk_idx[(int64_t)t * p.k + lane] : -1;
        if (idx >= p.E) idx = -1;
        const float ls = idx >= 0 ? open_logit(to_f32(row[idx])) : -INFINITY;
        const float dw = idx >= 0 ? p.d_weights[(int64_t)t * p.k + lane] * p.scale : 0.0f;
        const bool on = ls > -INFINITY;
        float add = 0.0f, dot = 0.0f;   // gradient of slot `lane`'s logit; what every logit gets times its probability
        if (p.renorm) {
            const float top = warp_max(ls);
            float v = !on ? 0.0f : p.sigmoid ? sigmoid_scaled(ls, fminf(top, 0.0f)) : expf(ls - top);
            const float sum = warp_sum(v);
            v = sum > 0.0f ? v / sum : 0.0f;
            add = v * (dw - warp_sum(v * dw));
            if (p.sigmoid && on) add /= 1.0f + expf(ls);
        } else if (p.sigmoid) {
            if (on) {
                const float v = sigmoid_scaled(ls, 0.0f);
                add = v * dw / (1.0f + expf(ls));
            }
        } else if (real) {
            const float v = on ? expf(ls - m) * inv : 0.0f;
            dot = warp_sum(v * dw);
            add = v * dw;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) d[i] -= q[i] * dot;
        for (int j = 0; j < p.k; ++j) {
            const int e = __shfl_sync(kAll, idx, j);
            const float v = __shfl_sync(kAll, add, j);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (e == lane + 32 * i) d[i] += v;
        }
    }
    L *out = static_cast<L *>(p.d_logits) + (int64_t)t * p.ld_d;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E) out[e] = from_f32<L>(d[i]);
    }
}

bool valid(const moe_router_config *c) {
    if (!c || c->num_experts < 1 || c->num_experts > 1024) return false;
    if (c->topk < 1 || c->topk > 32 || c->topk > c->num_experts) return false;
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return false;
    if (!valid_dtype(c->logits_dtype)) return false;
    if (!isfinite(c->weight_scale) || !isfinite(c->balance_coef) || !isfinite(c->z_coef)) return false;
    return c->score == MOE_SCORE_SOFTMAX || c->z_coef == 0.0f;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

int loss_warps(int T) { return std::min(std::max(T, 1), kMaxLossWarps); }

// Carves the workspace; returns its size.
size_t carve(int E, int T, int S, char *base, Partials *out) {
    const size_t rows = (size_t)loss_warps(T) + S;
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
    p.seq_bal = reinterpret_cast<float *>(take((size_t)S * 4));
    p.seq_z = reinterpret_cast<float *>(take((size_t)S * 4));
    if (out) *out = p;
    return o;
}

template <class L, int NI>
void launch_router(const RouterParams &p, bool loss, bool given, int warps, cudaStream_t s) {
    const int ctas = (warps + kWarpsPerCta - 1) / kWarpsPerCta;
    if (!loss) router_kernel<L, NI, false, false><<<ctas, kThreads, 0, s>>>(p);
    else if (given) router_kernel<L, NI, true, true><<<ctas, kThreads, 0, s>>>(p);
    else router_kernel<L, NI, true, false><<<ctas, kThreads, 0, s>>>(p);
}

// Calls f with the number of experts per lane as a template argument.
template <class F>
void by_experts(int E, F f) {
    if (E <= 32) f.template run<1>();
    else if (E <= 64) f.template run<2>();
    else if (E <= 128) f.template run<4>();
    else if (E <= 256) f.template run<8>();
    else if (E <= 512) f.template run<16>();
    else f.template run<32>();
}

struct RunRouter {
    const RouterParams &p;
    bool bf, loss, given;
    int warps;
    cudaStream_t s;
    template <int NI>
    void run() const {
        if (bf) launch_router<bf16, NI>(p, loss, given, warps, s);
        else launch_router<float, NI>(p, loss, given, warps, s);
    }
};

struct RunBwd {
    const RouterBwd &p;
    bool bf;
    cudaStream_t s;
    template <int NI>
    void run() const {
        const int ctas = (p.T + kWarpsPerCta - 1) / kWarpsPerCta;
        if (bf) router_bwd_kernel<bf16, NI><<<ctas, kThreads, 0, s>>>(p);
        else router_bwd_kernel<float, NI><<<ctas, kThreads, 0, s>>>(p);
    }
};

bool loss_ok(const moe_balance_io *l, const void *ws) {
    return l->num_seqs >= 1 && (l->seq_offsets || l->num_seqs == 1) && l->loss && l->counts && l->prob_mean &&
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
    p.scale = cfg->weight_scale;
    p.S = loss ? loss->num_seqs : 1;
    p.seq_offsets = loss ? loss->seq_offsets : nullptr;
    p.chunk = loss ? (T + loss_warps(T) - 1) / loss_warps(T) : 1;
    if (loss) carve(p.E, T, p.S, static_cast<char *>(ws), &p.part);
    if (T > 0) {
        by_experts(p.E, RunRouter{p, cfg->logits_dtype == MOE_DTYPE_BF16, loss != nullptr, given,
                                  (T + p.chunk - 1) / p.chunk, s});
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (loss) {
        SumParams q{p.part, p.seq_offsets, loss->counts, loss->prob_mean, loss->seq_tokens, T, p.E, p.k, p.S,
                    std::max(p.chunk, 1)};
        router_seq_kernel<<<p.S, kThreads, 0, s>>>(q);
        router_loss_kernel<<<1, 32, 0, s>>>(p.part, p.S, loss->seq_tokens, cfg->balance_coef, cfg->z_coef, loss->loss);
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_workspace_bytes(const moe_router_config *cfg, int max_tokens, int max_seqs) {
    if (!valid(cfg) || max_tokens < 0 || max_seqs < 1) return 0;
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
    if (d_loss && (!loss || loss->num_seqs < 1 || (!loss->seq_offsets && loss->num_seqs != 1) || !loss->counts ||
                   !loss->seq_tokens))
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
    by_experts(p.E, RunBwd{p, cfg->logits_dtype == MOE_DTYPE_BF16, static_cast<cudaStream_t>(stream)});
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
