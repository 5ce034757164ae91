"""The operators of an MoE block around the expert layer: cases, plain forms, calls and exact values.

Four operators, each in a plain form of elementary torch operations in 32 bits and as the calls a user makes of
moe_expert_ffn_gb300 (`own = True`):

  norm      the norms after one block and before the next, fused with the gate, the residual sum and the expert
            layer's input quantisation (moe.BlockNorm), forward and backward
  route     the top-k router (moe.Router.forward)
  balance   the balance and z losses with per-sequence expert counts, forward and gradient, together with the
            router's own (moe.Router.forward_train, .balance_loss, .backward)
  linear    products of 1 to 16 tokens with E2M1 weights under UE8M0 scales per 32 (moe.Fp4Linear)

The sizes are those of the package's workloads (hidden 7168 and 4096, inter 2048 and 14336, 256 and 8 experts, top-8 and
top-2, batches of 32 to 4096 tokens), with odd ones beside them.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
FLT_MAX = torch.finfo(torch.float32).max
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases -----------------------------------------------------------------
def _norm(name, T, H, **kw):
    case = {"name": name, "op": "norm", "T": T, "H": H, "stream": "bf16", "param": "f32", "gate": "channel", "post": True,
            "pre": True, "normed": True, "quant": "fp8", "residual_scale": 1.0, "backward": False}
    return {**case, **kw}


def _route(name, op, T, E, k, **kw):
    case = {"name": name, "op": op, "T": T, "E": E, "k": k, "logits": "f32", "score": "softmax", "renorm": True, "bias": False,
            "empty": 0, "zipf": False}
    if op == "balance":
        case.update(S=1, given=False)
    return {**case, **kw}


def _linear(name, M, N, K, **kw):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "act": "none", "add": False, "out": "bf16", **kw}


def listed():
    return [
        # one decoded token between two blocks: the call is all latency
        _norm("norm_token", 1, 7168, normed=True),
        # the prefill batch between two blocks: the stream, the router's input and the FP8 layer's input in one pass
        _norm("norm_prefill", 4096, 7168),
        # the FP4 layer's input format, a per-token gate, bf16 parameters, an odd batch
        _norm("norm_fp4_input", 1023, 4096, quant="ue8m0", gate="token", param="bf16", normed=False, residual_scale=0.5),
        # a training batch's backward pass of the same
        _norm("norm_backward", 4096, 7168, backward=True, quant="none"),
        # a float32 stream of a width that no vector divides, no post norm (pre-norm blocks), backward
        _norm("norm_backward_odd", 1777, 1001, backward=True, quant="none", stream="f32", post=False, gate="token"),
        # the router of a decode batch
        _route("route_decode", "route", 128, 256, 8),
        # the router of a long prefill, sigmoid scores, a selection bias, some experts closed, bf16 logits
        _route("route_prefill", "route", 32767, 256, 8, score="sigmoid", bias=True, empty=16, logits="bf16"),
        # a training batch of ragged sequences: routing, losses, counts and the gradient of the logits
        _route("balance_train", "balance", 65536, 256, 8, S=17, zipf=True),
        # a small batch routed elsewhere: losses and gradient for the given choice, few experts
        _route("balance_given", "balance", 2048, 8, 2, given=True, logits="bf16"),
        # a shared expert's gate and up product for one decoded token
        _linear("linear_token_swiglu", 1, 4096, 7168, act="swiglu"),
        # its down product for a few tokens, added to the routed experts' output
        _linear("linear_down_add", 5, 7168, 2048, add=True),
        # the widest product of the workloads for the most tokens
        _linear("linear_wide", 16, 28672, 4096, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "balance", "linear"])
    if op == "norm":
        quant = rng.choice(["none", "fp8", "ue8m0"])
        backward = rng.random() < 0.4
        H = rng.choice([4096, 7168, 128 * (2 * rng.randrange(0, 28) + 1)])
        if quant == "none" and rng.random() < 0.5:
            H = _log(rng, 33, 7000) | 1
        post = rng.random() < 0.7
        case = _norm("", _log(rng, 1, 4000) | 1, H, stream=rng.choice(["bf16", "bf16", "f32"]), param=rng.choice(["f32", "bf16"]),
                     gate=rng.choice(["none", "channel", "token"]), post=post, pre=True if quant != "none" else rng.random() < 0.8,
                     normed=True, quant="none" if backward else quant, residual_scale=rng.choice([1.0, 0.5, 0.25]),
                     backward=backward)
        if case["stream"] == "f32":
            case["T"] = max(1, case["T"] // 2) | 1
    elif op == "linear":
        act = rng.choice(["none", "swiglu"])
        K = 32 * (2 * _log(rng, 1, 111) + 1)
        n = min(_log(rng, 40, 14000), 28672 * 4096 // (2 * K))
        N = 2 * (n | 1) if act == "swiglu" else rng.choice([2 * (n | 1), n | 1])
        case = _linear("", rng.randint(1, 16), N, K, act=act, add=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    else:
        E = rng.choice([8, 256, _log(rng, 2, 1000) | 1])
        T = min(_log(rng, 1, 60000), 65536 * 256 // E) | 1
        case = _route("", op, T, E, rng.randint(1, min(E, 16)), logits=rng.choice(["f32", "bf16"]),
                      score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7, bias=rng.random() < 0.5,
                      empty=rng.choice([0, E // 8]), zipf=rng.random() < 0.5)
        if op == "balance":
            case.update(S=_log(rng, 1, 40), given=rng.random() < 0.3)
    del case["name"]
    return case


# ---- inputs ----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1_000_003 * int(seed) + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _inputs_norm(c, g):
    T, H, ty, pt = c["T"], c["H"], DTYPES[c["stream"]], DTYPES[c["param"]]
    d = {}
    chan = 1.0 + 4.0 * (torch.rand(H, generator=g, device=DEVICE) < 0.02)      # a stream has a few large channels
    d["residual"] = (_randn(g, T, H) * chan).to(ty)
    d["y"] = (0.5 * _randn(g, T, H)).to(ty)
    if T > 8:                                                                  # a padding token
        d["residual"][T // 2] = 0
        d["y"][T // 2] = 0
    d["w_post"] = (1.0 + 0.1 * _randn(g, H)).to(pt) if c["post"] else None
    d["w_pre"] = (1.0 + 0.1 * _randn(g, H)).to(pt) if c["pre"] else None
    d["gate"] = {"none": lambda: None, "channel": lambda: (0.3 * _randn(g, H)).to(pt),
                 "token": lambda: torch.sigmoid(_randn(g, T)).to(pt)}[c["gate"]]()
    if c["backward"]:
        # what the forward pass left: the stream after the block and the norms' reciprocal roots
        yf, rf = d["y"].float(), d["residual"].float()
        r1 = torch.rsqrt(yf.square().mean(1) + EPS) if c["post"] else None
        u = yf * r1[:, None] * d["w_post"].float() if c["post"] else yf
        gt = 1.0 if d["gate"] is None else d["gate"].float() if c["gate"] == "channel" else d["gate"].float()[:, None]
        d["h"] = (c["residual_scale"] * rf + gt * u).to(ty)
        d["rstd_post"] = r1
        d["rstd_pre"] = torch.rsqrt(d["h"].float().square().mean(1) + EPS) if c["pre"] else None
        d["dh"] = (1e-2 * _randn(g, T, H)).to(ty)
        d["dn"] = (1e-2 * _randn(g, T, H)).to(ty) if c["pre"] else None
        del d["residual"]
    return d


def _offsets(T, S, g):
    """Ragged sequences, some of them empty, over most of the batch."""
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEVICE).sort().values
    if S > 3:
        cut[S // 2] = cut[S // 2 - 1]
    zero = torch.zeros(1, dtype=cut.dtype, device=DEVICE)
    return torch.cat([zero, cut, torch.full_like(zero, T)]).to(torch.int32)


def _inputs_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(g, T, E)
    if c["zipf"]:
        rank = torch.empty(E, device=DEVICE)
        rank[torch.randperm(E, generator=g, device=DEVICE)] = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32)
        logits -= 1.2 * rank.log()
    if c["empty"]:
        logits[:, torch.randperm(E, generator=g, device=DEVICE)[: c["empty"]]] = -math.inf
    if T > 8:
        logits[T // 2] = -math.inf                                             # a padding token
    d = {"logits": logits.to(DTYPES[c["logits"]]), "bias": 0.1 * _randn(g, E) if c["bias"] else None}
    if c["op"] == "balance":
        d["seq_offsets"] = _offsets(T, c["S"], g) if c["S"] > 1 else None
        d["d_loss"] = torch.ones((), device=DEVICE)
        if c["given"]:
            idx = torch.rand(T, E, generator=g, device=DEVICE).topk(k, dim=1).indices
            idx[T // 2, k - 1] = -1                                            # an inactive slot
            d["topk_idx"] = idx.to(torch.int32)
        else:
            d["d_weights"] = 1e-3 * _randn(g, T, k)
    return d


def _inputs_linear(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    n_out = N // 2 if c["act"] == "swiglu" else N
    w = torch.randint(0, 256, (N, K // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    # scales of weights ~ N(0, 1/K) quantised to E2M1: exponents around log2(3 / sqrt(K) / 6)
    mid = 127 + round(math.log2(0.5 / math.sqrt(K)))
    w_sf = (mid + torch.randint(-1, 2, (N, K // 32), generator=g, device=DEVICE)).to(torch.uint8)
    d = {"x": _randn(g, M, K).to(torch.bfloat16), "w": w, "w_sf": w_sf}
    d["add"] = _randn(g, M, n_out).to(DTYPES[c["out"]]) if c["add"] else None
    return d


def _inputs(case, seed):
    g = _gen(seed)
    return {"norm": _inputs_norm, "route": _inputs_route, "balance": _inputs_route, "linear": _inputs_linear}[case["op"]](case, g)


Z_COEF, BALANCE_COEF = 1e-3, 1e-2


def _coefs(c):
    """The z loss belongs to softmax scores."""
    return BALANCE_COEF, (Z_COEF if c["score"] == "softmax" else 0.0)


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if own:
        import moe_expert_ffn_gb300 as moe
        c = case
        if c["op"] == "norm":
            op = moe.BlockNorm(c["H"], eps=EPS, residual_scale=c["residual_scale"], gate=None if c["gate"] == "none" else c["gate"],
                               quant=None if c["quant"] == "none" else c["quant"], dtype=DTYPES[c["stream"]],
                               param_dtype=DTYPES[c["param"]], device=DEVICE)
            if c["backward"]:
                s["out"] = op.grad_buffers(c["T"], block=True, post=c["post"])
            else:
                s["out"] = op.buffers(c["T"], block=True, post=c["post"], pre=c["pre"], normed=c["normed"] and c["pre"])
        elif c["op"] == "linear":
            op = moe.Fp4Linear(c["K"], c["N"], act=None if c["act"] == "none" else c["act"], out_dtype=DTYPES[c["out"]], device=DEVICE)
            op.transform_weights(s["w"], s["w_sf"])
            s["out"] = op.buffers(c["M"])
        else:
            bal, z = _coefs(c) if c["op"] == "balance" else (0.0, 0.0)
            op = moe.Router(c["E"], c["k"], score=c["score"], renormalize=c["renorm"], balance_coef=bal, z_coef=z,
                            logits_dtype=DTYPES[c["logits"]], max_tokens=c["T"], max_seqs=c.get("S", 1), device=DEVICE)
            s["out"] = op.buffers(c["T"], num_seqs=c.get("S", 1)) if c["op"] == "balance" else op.buffers(c["T"])
            s["d_logits"] = torch.empty_like(s["logits"]) if c["op"] == "balance" else None
        s["op"] = op
    return s


# ---- plain forms -----------------------------------------------------------
def _gate(c, gate):
    if gate is None:
        return 1.0
    return gate.float() if c["gate"] == "channel" else gate.float()[:, None]


def _quantise(v, quant):
    """[T, H] -> E4M3 values and their scales: amax/448 per 128, or the power of two at or above it per 32."""
    T, H = v.shape
    if quant == "fp8":
        g = v.view(T, H // 128, 128)
        sf = g.abs().amax(2) / 448.0
        div = torch.where(sf > 0, sf, torch.ones_like(sf))
        return (g / div[:, :, None]).view(T, H).to(torch.float8_e4m3fn), sf
    g = v.view(T, H // 32, 32)
    ratio = g.abs().amax(2) / 448.0
    m, e = torch.frexp(ratio)
    e = torch.where(ratio > 0, torch.where(m == 0.5, e - 1, e), torch.full_like(e, -127)).clamp(-127, 127)
    q = torch.ldexp(g, -e[:, :, None]).view(T, H).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm(s):
    c = s["case"]
    y, ty, out = s["y"].float(), s["y"].dtype, {}
    u = y
    if c["post"]:
        r1 = torch.rsqrt(y.square().mean(1) + EPS)
        out["rstd_post"] = r1
        u = y * r1[:, None] * s["w_post"].float()
    h = c["residual_scale"] * s["residual"].float() + _gate(c, s["gate"]) * u
    out["h"] = h.to(ty)
    if c["pre"]:
        r2 = torch.rsqrt(h.square().mean(1) + EPS)
        v = h * r2[:, None] * s["w_pre"].float()
        out["rstd_pre"] = r2
        if c["normed"]:
            out["n"] = v.to(ty)
        if c["quant"] != "none":
            out["codes"], out["sf"] = _quantise(v, c["quant"])
    return out


def _plain_norm_backward(s):
    c = s["case"]
    h, y, ty, out = s["h"].float(), s["y"].float(), s["y"].dtype, {}
    D = s["dh"].float()
    if c["pre"]:
        dn, r2 = s["dn"].float(), s["rstd_pre"][:, None]
        hat = h * r2
        a = dn * s["w_pre"].float()
        out["dw_pre"] = (dn * hat).sum(0)
        D = D + r2 * (a - hat * (a * hat).mean(1, keepdim=True))
    out["dresidual"] = (c["residual_scale"] * D).to(ty)
    gate = _gate(c, s["gate"])
    Dg = D * gate
    u = y
    if c["post"]:
        r1 = s["rstd_post"][:, None]
        hat = y * r1
        u = hat * s["w_post"].float()
        b = Dg * s["w_post"].float()
        out["dw_post"] = (Dg * hat).sum(0)
        out["dy"] = (r1 * (b - hat * (b * hat).mean(1, keepdim=True))).to(ty)
    else:
        out["dy"] = Dg.to(ty)
    if s["gate"] is not None:
        out["dgate"] = (D * u).sum(0 if c["gate"] == "channel" else 1)
    return out


def _choose(c, L, bias):
    """Top-k of logit + bias, ties to the lowest index; -1 where nothing is left to choose."""
    key = L if bias is None else L + bias
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, : c["k"]], idx[:, : c["k"]]
    return torch.where(val > -math.inf, idx, torch.full_like(idx, -1))


def _finite(logits):
    L = logits.float()
    return torch.where(torch.isnan(L), torch.full_like(L, -math.inf), L).clamp(max=FLT_MAX)


def _scores(c, L):
    """softmax, or sigmoid"""
    if c["score"] == "sigmoid":
        return torch.sigmoid(L)
    m = L.amax(1, keepdim=True)
    e = torch.exp(L - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _weights(c, p, idx):
    on = idx >= 0
    w = torch.where(on, torch.gather(p, 1, idx.clamp(min=0)), torch.zeros_like(p[:, :1]))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    return w, on


def _plain_route(s):
    c = s["case"]
    L = _finite(s["logits"])
    idx = _choose(c, L, s["bias"])
    w, _ = _weights(c, _scores(c, L), idx)
    return {"topk_idx": idx.to(torch.int32), "topk_weights": w}


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    bal, z = _coefs(c)
    L = _finite(s["logits"])
    real = (L > -math.inf).any(1)
    p = _scores(c, L)
    out = {}
    idx = s["topk_idx"].long() if c["given"] else _choose(c, L, s["bias"])
    on = idx >= 0
    picked = torch.zeros(T, E + 1, device=L.device).scatter_(1, torch.where(on, idx, torch.full_like(idx, E)), 1.0)[:, :E]
    # which sequence a token is in, as rows of a [S, T] indicator
    at = torch.arange(T, device=L.device)
    off = s["seq_offsets"] if s["seq_offsets"] is not None else torch.tensor([0, T], device=L.device)
    seq = ((at[None] >= off[:-1, None]) & (at[None] < off[1:, None]) & real[None]).float()
    n = seq.sum(1)
    q = p if c["score"] == "softmax" else p / p.sum(1, keepdim=True).clamp(min=1e-30)
    counts, mean = seq @ picked, (seq @ q) / n.clamp(min=1)[:, None]
    f = E * counts / (k * n.clamp(min=1)[:, None])
    seqs, total = (n > 0).sum().clamp(min=1).float(), n.sum().clamp(min=1)
    inside = seq.sum(0)
    l_bal = bal * (f * mean).sum() / seqs
    m = torch.where(real, L.amax(1), torch.zeros(T, device=L.device))
    lse = torch.where(real, m + torch.log(torch.exp(L - m[:, None]).sum(1).clamp(min=1e-30)), torch.zeros_like(m))
    l_z = z * (lse.square() * inside).sum() / total
    # gradient: the losses' and the weights'
    C = seq.t() @ (bal * f / (seqs * n.clamp(min=1)[:, None]))
    d = q * (C - (q * C).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1 - p)
    else:
        d = d + (2 * z / total * lse * inside)[:, None] * q
    d = d * s["d_loss"]
    if not c["given"]:
        w, _ = _weights(c, p, idx)
        out["topk_idx"], out["topk_weights"] = idx.to(torch.int32), w
        G = torch.zeros(T, E + 1, device=L.device).scatter_(1, torch.where(on, idx, torch.full_like(idx, E)), s["d_weights"])[:, :E]
        if c["renorm"]:
            W = torch.zeros(T, E + 1, device=L.device).scatter_(1, torch.where(on, idx, torch.full_like(idx, E)), w)[:, :E]
            dg = W * (G - (W * G).sum(1, keepdim=True))
            d = d + (dg * (1 - p) if c["score"] == "sigmoid" else dg)
        elif c["score"] == "sigmoid":
            d = d + G * p * (1 - p)
        else:
            d = d + p * (G - (p * G).sum(1, keepdim=True))
    out.update(loss=torch.stack([l_bal + l_z, l_bal, l_z]), counts=counts.round().to(torch.int32), prob_mean=mean,
               seq_tokens=n.round().to(torch.int32), d_logits=d.to(s["logits"].dtype))
    return out


def _plain_linear(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    lut = torch.tensor(E2M1, device=s["w"].device)
    val = torch.stack([lut[(s["w"] & 15).long()], lut[(s["w"] >> 4).long()]], 2).view(N, K // 32, 32)
    W = torch.ldexp(val, (s["w_sf"].to(torch.int32) - 127)[:, :, None]).view(N, K)
    y = s["x"].float() @ W.t()
    if c["act"] == "swiglu":
        g, u = y[:, : N // 2], y[:, N // 2:]
        y = g * torch.sigmoid(g) * u
    if s["add"] is not None:
        y = y + s["add"].float()
    return {"y": y.to(DTYPES[c["out"]])}


# ---- the calls -------------------------------------------------------------
def _own_norm(s):
    c, op = s["case"], s["op"]
    o = op.forward(s["residual"], s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], out=s["out"])
    out = {"h": o.h}
    if c["post"]:
        out["rstd_post"] = o.rstd_post
    if c["pre"]:
        out["rstd_pre"] = o.rstd_pre
        if c["normed"]:
            out["n"] = o.n
        if c["quant"] != "none":
            out["codes"] = o.codes.view(torch.float8_e4m3fn)
            out["sf"] = o.sf if c["quant"] == "fp8" else o.sf.view(torch.float8_e8m0fnu)
    return out


def _own_norm_backward(s):
    c, op = s["case"], s["op"]
    o = op.backward(s["h"], s["dh"], s["dn"], y=s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                    rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], out=s["out"])
    out = {"dresidual": o.dresidual, "dy": o.dy}
    if c["pre"]:
        out["dw_pre"] = o.dw_pre
    if c["post"]:
        out["dw_post"] = o.dw_post
    if s["gate"] is not None:
        out["dgate"] = o.dgate
    return out


def _own_route(s):
    o = s["op"].forward(s["logits"], s["bias"], out=s["out"])
    return {"topk_idx": o.topk_idx, "topk_weights": o.topk_weights}


def _own_balance(s):
    c, op = s["case"], s["op"]
    if c["given"]:
        o = op.balance_loss(s["logits"], s["topk_idx"], s["seq_offsets"], out=s["out"])
        out = {}
    else:
        o = op.forward_train(s["logits"], s["bias"], s["seq_offsets"], out=s["out"])
        out = {"topk_idx": o.topk_idx, "topk_weights": o.topk_weights}
    d = op.backward(s["logits"], o, d_weights=s.get("d_weights"), d_loss=s["d_loss"], seq_offsets=s["seq_offsets"], out=s["d_logits"])
    out.update(loss=o.loss, counts=o.counts, prob_mean=o.prob_mean, seq_tokens=o.seq_tokens, d_logits=d)
    return out


def _own_linear(s):
    return {"y": s["op"].forward(s["x"], add=s["add"], out=s["out"])}


def run(state):
    c = state["case"]
    kind = c["op"] if c["op"] != "norm" or not c["backward"] else "norm_backward"
    if own:
        return {"norm": _own_norm, "norm_backward": _own_norm_backward, "route": _own_route, "balance": _own_balance,
                "linear": _own_linear}[kind](state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route, "balance": _plain_balance,
            "linear": _plain_linear}[kind](state)


# ---- work ------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        T, H, es, ps = c["T"], c["H"], SIZE[c["stream"]], SIZE[c["param"]]
        par = ps * (H * (c["post"] + c["pre"]) + {"none": 0, "channel": H, "token": T}[c["gate"]]) + 4 * T * (c["post"] + c["pre"])
        if c["backward"]:  # y, dh in; dresidual, dy out; with the pre norm h and dn in
            sums = 4 * (H * (c["post"] + c["pre"]) + {"none": 0, "channel": H, "token": T}[c["gate"]])
            return {"bytes": T * H * es * (4 + 2 * c["pre"]) + par + sums, "flops": T * H * (8 + 10 * c["pre"] + 10 * c["post"])}
        out = es * (1 + (c["normed"] and c["pre"])) + {"none": 0, "fp8": 1 + 4 / 128, "ue8m0": 1 + 1 / 32}[c["quant"]]
        return {"bytes": int(T * H * (2 * es + out)) + par, "flops": T * H * (4 + 4 * c["post"] + 4 * c["pre"] + 3 * (c["quant"] != "none"))}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * SIZE[c["logits"]] + 8 * T * k + (4 * E if c["bias"] else 0), "flops": T * (4 * E + 4 * k)}
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        idx = 4 * T * k if c["given"] else 12 * T * k
        return {"bytes": 2 * T * E * SIZE[c["logits"]] + idx + 8 * S * E + 8 * S + 16, "flops": T * (14 * E + 8 * k)}
    M, N, K = c["M"], c["N"], c["K"]
    n_out = N // 2 if c["act"] == "swiglu" else N
    return {"bytes": N * K // 2 + N * K // 32 + 2 * M * K + M * n_out * SIZE[c["out"]] * (1 + c["add"]), "flops": 2 * M * N * K}


# ---- exact values ----------------------------------------------------------
def _to_grid(v):
    """Nearest E4M3 value, ties to even, by arithmetic on the exponent: 3 fraction bits, smallest step 2^-9, largest 448."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 4).clamp(min=-9))
    return torch.sign(v) * torch.round(a / step) * step


def _exact_norm(c, d):
    f = {n: t.double() for n, t in d.items() if t is not None}
    out = {}
    u = f["y"]
    if c["post"]:
        out["rstd_post"] = (f["y"].pow(2).sum(1) / c["H"] + EPS).pow(-0.5)
        u = torch.einsum("th,t,h->th", f["y"], out["rstd_post"], f["w_post"])
    if d["gate"] is not None:
        u = u * (f["gate"] if c["gate"] == "channel" else f["gate"].unsqueeze(1))
    out["h"] = f["residual"] * c["residual_scale"] + u
    if c["pre"]:
        h = out["h"]                                           # the norm reads the sum before it is rounded to the stream's type
        out["rstd_pre"] = (h.pow(2).sum(1) / c["H"] + EPS).pow(-0.5)
        v = torch.einsum("th,t,h->th", h, out["rstd_pre"], f["w_pre"])
        if c["normed"]:
            out["n"] = v
        if c["quant"] != "none":
            G = 128 if c["quant"] == "fp8" else 32
            top = v.reshape(c["T"], -1, G).abs().max(2).values
            sf = top / 448 if c["quant"] == "fp8" else torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-127))
            each = sf.repeat_interleave(G, 1)
            out["codes"] = _to_grid(torch.where(each > 0, v / each, torch.zeros_like(v)))
            out["sf"] = sf
    return out


def _exact_norm_backward(c, d):
    f = {n: t.double() for n, t in d.items() if t is not None}
    H, out = c["H"], {}
    total = f["dh"]
    if c["pre"]:
        r = f["rstd_pre"].unsqueeze(1)
        a = f["dn"] * f["w_pre"]
        out["dw_pre"] = torch.einsum("th,th,t->h", f["dn"], f["h"], f["rstd_pre"])
        total = total + r * a - r.pow(3) * f["h"] * ((a * f["h"]).sum(1, keepdim=True) / H)
    out["dresidual"] = total * c["residual_scale"]
    inner = total
    if d["gate"] is not None:
        inner = total * (f["gate"] if c["gate"] == "channel" else f["gate"].unsqueeze(1))
    branch = f["y"]
    if c["post"]:
        r = f["rstd_post"].unsqueeze(1)
        out["dw_post"] = torch.einsum("th,th,t->h", inner, f["y"], f["rstd_post"])
        b = inner * f["w_post"]
        out["dy"] = r * b - r.pow(3) * f["y"] * ((b * f["y"]).sum(1, keepdim=True) / H)
        branch = f["y"] * r * f["w_post"]
    else:
        out["dy"] = inner
    if d["gate"] is not None:
        out["dgate"] = torch.einsum("th,th->h" if c["gate"] == "channel" else "th,th->t", total, branch)
    return out


def _exact_route(c, d, grads):
    T, E, k = c["T"], c["E"], c["k"]
    x = torch.nan_to_num(d["logits"].double(), nan=-math.inf, posinf=FLT_MAX, neginf=-math.inf)
    # the choice is made on 32-bit keys, so it is taken from them: the k largest by (key, -index)
    if c.get("given"):
        idx = d["topk_idx"].long()
    else:
        key = x.float() if d["bias"] is None else x.float() + d["bias"]
        order = torch.argsort(-key, dim=1, stable=True)[:, :k]
        idx = order.masked_fill(torch.gather(key, 1, order) == -math.inf, -1)
    hit = torch.nn.functional.one_hot(idx + 1, E + 1)[:, :, 1:].sum(1).double() if T * k * E < 3e8 else _hits(idx, E)
    valid = torch.isfinite(x).any(1)
    safe = torch.where(valid.unsqueeze(1), x, torch.zeros_like(x))
    lse = torch.logsumexp(safe, 1)
    if c["score"] == "softmax":
        raw = torch.exp(safe - lse.unsqueeze(1)) * valid.unsqueeze(1)
        share, slope = raw, torch.ones_like(raw)
    else:
        raw = torch.special.expit(x)
        share = raw / raw.sum(1, keepdim=True).clamp(min=1e-300)
        slope = 1 - raw
    sel = raw * hit
    top = sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if c["renorm"] else sel
    out = {}
    if not c.get("given"):
        out["topk_idx"] = None
        out["topk_weights"] = torch.gather(top, 1, idx.clamp(min=0)) * (idx >= 0)
    if not grads:
        return out
    off = d["seq_offsets"].tolist() if d["seq_offsets"] is not None else [0, T]
    bal, z = _coefs(c)
    spans = [(a, b) for a, b in zip(off[:-1], off[1:])]
    n = [int(valid[a:b].sum()) for a, b in spans]
    used, tokens = max(1, sum(v > 0 for v in n)), max(1, sum(n))
    mean, l_bal, l_z = torch.zeros(len(n), E, dtype=torch.float64, device=x.device), 0.0, 0.0
    g = torch.zeros_like(x)
    for i, (a, b) in enumerate(spans):
        if n[i] == 0:
            continue
        on = valid[a:b].unsqueeze(1)
        mean[i] = (share[a:b] * on).sum(0) / n[i]
        load = (hit[a:b] * on).sum(0) * (E / (k * n[i]))
        l_bal = l_bal + bal * (load * mean[i]).sum() / used
        pull = load * (bal / used / n[i])
        g[a:b] += share[a:b] * slope[a:b] * (pull - (share[a:b] * pull).sum(1, keepdim=True)) * on
        if z:
            l_z = l_z + z * (lse[a:b].pow(2) * on[:, 0]).sum() / tokens
            g[a:b] += (2 * z / tokens) * lse[a:b].unsqueeze(1) * share[a:b] * on
    g = g * d["d_loss"].double()
    if not c.get("given"):
        G = torch.zeros(T, E + 1, dtype=torch.float64, device=x.device)
        G.scatter_add_(1, torch.where(idx >= 0, idx, E), d["d_weights"].double())
        G = G[:, :E]
        if c["renorm"] or c["score"] == "softmax":
            base = top if c["renorm"] else raw
            g = g + base * slope * (G - (base * G).sum(1, keepdim=True))
        else:
            g = g + G * raw * slope
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    l_bal, l_z = l_bal + zero, l_z + zero
    out.update(loss=torch.stack([l_bal + l_z, l_bal, l_z]), counts=None, prob_mean=mean, seq_tokens=None, d_logits=g)
    return out


def _hits(idx, E):
    hit = torch.zeros(idx.shape[0], E + 1, dtype=torch.float64, device=idx.device)
    for j in range(idx.shape[1]):
        hit.scatter_add_(1, (idx[:, j:j + 1] + 1), torch.ones(idx.shape[0], 1, dtype=torch.float64, device=idx.device))
    return hit[:, 1:]


def _exact_linear(c, d):
    N, K = c["N"], c["K"]
    w = d["w"].cpu().numpy()
    nib = np.empty((N, K), dtype=np.uint8)
    nib[:, 0::2], nib[:, 1::2] = w & 15, w >> 4
    mag = nib & 7
    e, m = (mag >> 1).astype(np.int32), (mag & 1).astype(np.float64)
    val = np.where(e == 0, 0.5 * m, np.ldexp(1.0 + 0.5 * m, e - 1)) * np.where(nib & 8, -1.0, 1.0)
    val *= np.repeat(np.ldexp(1.0, d["w_sf"].cpu().numpy().astype(np.int32) - 127), 32, axis=1)
    y = d["x"].double() @ torch.from_numpy(val).to(d["x"].device).t()
    if c["act"] == "swiglu":
        a, b = y.chunk(2, 1)
        y = a / (1 + torch.exp(-a)) * b
    return {"y": y if d["add"] is None else y + d["add"].double()}


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] == "norm":
        return _exact_norm_backward(c, d) if c["backward"] else _exact_norm(c, d)
    if c["op"] == "linear":
        return _exact_linear(c, d)
    return _exact_route(c, d, c["op"] == "balance")
