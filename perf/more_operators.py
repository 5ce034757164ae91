"""The operators of a dense FP8 layer beside the routed experts, and routing within groups of experts: cases, plain forms,
calls and exact values.

Four operators, each in a plain form of elementary torch operations in 32 bits and as the calls a user makes of
moe_expert_ffn_gb300 (`own = True`):

  route     top-k routing limited to the best groups of experts (moe.Router with groups), alone and with losses and gradient
  linear    products of any number of tokens with E4M3 weights under f32 scales per 128 x 128, tokens with scales per
            1 x 128 (moe.Fp8Linear.forward), with SwiGLU and the next product's quantised input, or an added input
  grad      the gradients of the same for its input (.backward_input) and its weights (.backward_weight)
  quant     E4M3 codes with scales per 1 x 128 along rows, per 128 x 1 along columns, or both in one pass, of a tensor, of
            SwiGLU's output, or of SwiGLU's gradient; per 128 x 128 of weights (moe.Fp8Quant)

The sizes are those of the package's workloads (hidden 7168 and 4096, inter 2048 and 14336, 256 experts, top-8, batches of 1
to 4096 tokens), with odd ones beside them.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
FLT_MAX = torch.finfo(torch.float32).max
BALANCE_COEF = 1e-2


# ---- cases -----------------------------------------------------------------
def _route(name, T, E, k, **kw):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "groups": 8, "topk_groups": 4, "group_score": "top2",
            "logits": "f32", "score": "sigmoid", "bias": True, "train": False, "S": 1, "zipf": False, **kw}


def _linear(name, T, N, K, **kw):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "act": "none", "quant": False, "add": False, "out": "bf16", **kw}


def _grad(name, of, T, N, K, **kw):
    return {"name": name, "op": "grad", "of": of, "T": T, "N": N, "K": K, "add": False, "out": "f32" if of == "weight" else "bf16",
            **kw}


def _quant(name, kind, T, H, **kw):
    return {"name": name, "op": "quant", "kind": kind, "T": T, "H": H, "rows": True, "cols": True, "dtype": "bf16", **kw}


def listed():
    return [
        # the router of a decode batch: scores plus balancing biases, the best 4 of 8 groups by their two best experts
        _route("route_groups_decode", 128, 256, 8),
        # the router of a long prefill
        _route("route_groups_prefill", 32767, 256, 8, zipf=True),
        # a training batch of ragged sequences: softmax scores, groups by their best expert, losses and gradient
        _route("route_groups_train", 32768, 256, 8, groups=4, topk_groups=2, group_score="max", score="softmax", bias=False,
               train=True, S=17, logits="bf16"),
        # a shared expert's gate and up product for one decoded token, with the down product's input
        _linear("linear_token_swiglu", 1, 4096, 7168, act="swiglu", quant=True),
        # its down product for a decode batch, added to the routed experts' output
        _linear("linear_decode_add", 128, 7168, 2048, add=True),
        # the gate and up product of a prefill batch
        _linear("linear_prefill_swiglu", 4096, 4096, 7168, act="swiglu", quant=True),
        # an odd batch, sizes that end inside a block of 128 on both sides
        _linear("linear_odd", 999, 2064, 4176, out="f32"),
        # the widest dense layer of the workloads
        _linear("linear_wide", 2048, 28672, 4096),
        # the down product's input gradient of a training batch
        _grad("grad_input", "input", 4096, 7168, 2048),
        # the gate and up product's weight gradient, added to what earlier micro-batches left
        _grad("grad_weight", "weight", 4096, 4096, 7168, add=True),
        # the layer's input of a training batch, quantised for the forward product and for the weights' gradient
        _quant("quant_tokens", "plain", 4096, 7168),
        # SwiGLU's gradient of an odd batch, quantised for both gradients of the gate and up product
        _quant("quant_swiglu_grad", "swiglu_grad", 1777, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "linear", "linear", "grad", "grad", "quant"])
    if op == "route":
        groups, size = rng.choice([(8, 32), (4, 64), (8, 8), (2, 32), (16, 16), (8, 20), (rng.randint(2, 12), rng.randint(2, 40))])
        E = groups * size
        use = rng.randint(1, groups - 1)
        score, train = rng.choice(["softmax", "sigmoid", "sigmoid"]), rng.random() < 0.4
        case = _route("", min(_log(rng, 1, 40000), 32768 * 256 // E) | 1, E, rng.randint(1, min(use * size, 16)), groups=groups,
                      topk_groups=use, group_score=rng.choice(["max", "top2"]), score=score, bias=rng.random() < 0.6, train=train,
                      S=_log(rng, 1, 40) if train else 1, zipf=rng.random() < 0.5, logits=rng.choice(["f32", "bf16"]))
    elif op == "quant":
        kind = rng.choice(["plain", "swiglu", "swiglu_grad", "blocks"])
        H = 16 * _log(rng, 1, 900)
        if kind in ("swiglu", "swiglu_grad"):
            H = 128 * _log(rng, 1, 56)
        rows, cols = rng.choice([(True, False), (False, True), (True, True)])
        T = min(_log(rng, 1, 9000), 4096 * 7168 // H) | 1
        case = _quant("", kind, T, H, rows=rows or kind == "blocks", cols=cols and kind != "blocks",
                      dtype=rng.choice(["bf16", "bf16", "f32"]))
    else:
        T, most = _log(rng, 1, 9000), 2048 * 28672 * 4096
        K = 16 * _log(rng, 8, 600)
        N = 16 * _log(rng, 8, 600)
        if T * N * K > most:
            T = max(1, most // (N * K))
        if op == "grad":
            of = rng.choice(["input", "weight"])
            case = _grad("", of, T, N, K, add=rng.random() < 0.4)
            if of == "input":
                case["out"] = rng.choice(["bf16", "f32"])
        else:
            act = rng.choice(["none", "swiglu"])
            if act == "swiglu":
                N = 256 * max(1, N // 256)
            quant = act == "swiglu" and rng.random() < 0.6
            case = _linear("", T, N, K, act=act, quant=quant, add=not quant and rng.random() < 0.4,
                           out=rng.choice(["bf16", "f32"]))
    del case["name"]
    return case


# ---- inputs ----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1_000_003 * int(seed) + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _up(n, m=128):
    return (n + m - 1) // m


def _scaled(v, dims):
    """f32 [R, C] -> E4M3 codes and the scales amax / 448 of its blocks of dims[0] x dims[1] (0 where a block is zero)."""
    R, C = v.shape
    br, bc = dims
    p = torch.nn.functional.pad(v, (0, -C % bc, 0, -R % br))
    b = p.view(p.shape[0] // br, br, p.shape[1] // bc, bc)
    sf = b.abs().amax((1, 3)) / 448.0
    inv = torch.where(sf > 0, sf, torch.ones_like(sf)).reciprocal()
    q = (b * inv[:, None, :, None]).view(p.shape)[:R, :C].to(torch.float8_e4m3fn)
    return q.contiguous(), sf


def _coded(v, dims):
    q, sf = _scaled(v, dims)
    return q.view(torch.uint8), sf


def _offsets(T, S, g):
    """Ragged sequences over most of the batch."""
    cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEVICE).sort().values
    zero = torch.zeros(1, dtype=cut.dtype, device=DEVICE)
    return torch.cat([zero, cut, torch.full_like(zero, T)]).to(torch.int32)


def _inputs_route(c, g):
    T, E = c["T"], c["E"]
    logits = _randn(g, T, E)
    if c["zipf"]:
        rank = torch.empty(E, device=DEVICE)
        rank[torch.randperm(E, generator=g, device=DEVICE)] = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32)
        logits -= 0.5 * rank.log()
    if T > 8:
        logits[T // 2] = -math.inf                                             # a padding token
        logits[T // 3, : E // c["groups"]] = -math.inf                         # a token whose first group is closed
    d = {"logits": logits.to(DTYPES[c["logits"]]), "bias": 0.1 * _randn(g, E) if c["bias"] else None}
    if c["train"]:
        d["seq_offsets"] = _offsets(T, c["S"], g) if c["S"] > 1 else None
        d["d_loss"] = torch.ones((), device=DEVICE)
        d["d_weights"] = 1e-3 * _randn(g, T, c["k"])
    return d


def _tokens(g, T, H, scale=1.0):
    """Activations: tokens of different magnitude, a few large channels, and a padding token."""
    v = _randn(g, T, H) * torch.exp(0.5 * _randn(g, T, 1)) * scale
    v *= 1.0 + 4.0 * (torch.rand(H, generator=g, device=DEVICE) < 0.02)
    if T > 8:
        v[T // 2] = 0
    return v


def _inputs_linear(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    d = {}
    d["x"], d["x_sf"] = _coded(_tokens(g, T, K), (1, 128))
    d["w"], d["w_sf"] = _coded(_randn(g, N, K) / math.sqrt(K), (128, 128))
    n_out = N // 2 if c["act"] == "swiglu" else N
    d["add"] = _randn(g, T, n_out).to(DTYPES[c["out"]]) if c["add"] else None
    return d


def _inputs_grad(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    d = {}
    dy = _tokens(g, T, N, 1e-3)
    if c["of"] == "input":
        d["dy"], d["dy_sf"] = _coded(dy, (1, 128))
        d["w"], d["w_sf"] = _coded(_randn(g, N, K) / math.sqrt(K), (128, 128))
        d["add"] = (1e-3 * _randn(g, T, K)).to(DTYPES[c["out"]]) if c["add"] else None
    else:
        d["dy"], d["dy_sf"] = _coded(dy, (128, 1))
        d["x"], d["x_sf"] = _coded(_tokens(g, T, K), (128, 1))
        d["add"] = 1e-2 * _randn(g, N, K) if c["add"] else None
    return d


def _inputs_quant(c, g):
    T, H, ty = c["T"], c["H"], DTYPES[c["dtype"]]
    if c["kind"] == "blocks":
        return {"v": (_randn(g, T, H) / math.sqrt(H)).to(ty)}
    d = {"v": _tokens(g, T, H * (1 if c["kind"] == "plain" else 2)).to(ty)}
    if c["kind"] == "swiglu_grad":
        d["d"] = _tokens(g, T, H, 1e-3).to(ty)
    return d


def _inputs(case, seed):
    return {"route": _inputs_route, "linear": _inputs_linear, "grad": _inputs_grad, "quant": _inputs_quant}[case["op"]](case, _gen(seed))


def prepare(case, seed):
    c = case
    s = {"case": c, **_inputs(c, seed)}
    if own:
        import moe_expert_ffn_gb300 as moe
        T = c["T"]
        if c["op"] == "route":
            op = moe.Router(c["E"], c["k"], score=c["score"], balance_coef=BALANCE_COEF if c["train"] else 0.0,
                            logits_dtype=DTYPES[c["logits"]], max_tokens=T, max_seqs=c["S"], device=DEVICE,
                            bias_on="score" if c["score"] == "sigmoid" else "logit", groups=c["groups"],
                            topk_groups=c["topk_groups"], group_score=c["group_score"])
            s["out"] = op.buffers(T, num_seqs=c["S"]) if c["train"] else op.buffers(T)
            s["d_logits"] = torch.empty_like(s["logits"]) if c["train"] else None
        elif c["op"] == "quant":
            act = "swiglu" if c["kind"].startswith("swiglu") else None
            op = moe.Fp8Quant(c["H"], act=act, dtype=DTYPES[c["dtype"]], device=DEVICE)
            s["out"] = (op.weight_buffers(T) if c["kind"] == "blocks"
                        else op.buffers(T, rows=c["rows"], cols=c["cols"], grad=c["kind"] == "swiglu_grad"))
        else:
            op = moe.Fp8Linear(c["K"], c["N"], act=None if c.get("act", "none") == "none" else c["act"],
                               quant="fp8" if c.get("quant") else None, out_dtype=DTYPES[c["out"]], device=DEVICE)
            if c["op"] == "linear":
                s["out"] = op.buffers(T)
            else:
                s["out"] = op.input_grad_buffer(T) if c["of"] == "input" else op.weight_grad_buffer()
        s["op"] = op
    return s


# ---- plain forms -----------------------------------------------------------
def _spread(codes, sf, dims):
    """What the codes stand for, in f32."""
    R, C = codes.shape
    s = sf.repeat_interleave(dims[0], 0)[:R].repeat_interleave(dims[1], 1)[:, :C]
    return codes.view(torch.float8_e4m3fn).float() * s


def _silu(g):
    return g * torch.sigmoid(g)


def _plain_linear(s):
    c = s["case"]
    y = _spread(s["x"], s["x_sf"], (1, 128)) @ _spread(s["w"], s["w_sf"], (128, 128)).t()
    if c["act"] == "swiglu":
        y = _silu(y[:, : c["N"] // 2]) * y[:, c["N"] // 2:]
    if c["quant"]:
        q, sf = _scaled(y, (1, 128))
        return {"codes": q, "sf": sf}
    if s["add"] is not None:
        y = y + s["add"].float()
    return {"y": y.to(DTYPES[c["out"]])}


def _plain_grad(s):
    c = s["case"]
    if c["of"] == "input":
        r = _spread(s["dy"], s["dy_sf"], (1, 128)) @ _spread(s["w"], s["w_sf"], (128, 128))
    else:
        r = _spread(s["dy"], s["dy_sf"], (128, 1)).t() @ _spread(s["x"], s["x_sf"], (128, 1))
    if s["add"] is not None:
        r = r + s["add"].float()
    return {"d" + c["of"]: r.to(DTYPES[c["out"]])}


def _plain_quant(s):
    c = s["case"]
    H, v = c["H"], s["v"].float()
    if c["kind"] == "blocks":
        q, sf = _scaled(v, (128, 128))
        return {"codes": q, "sf": sf}
    if c["kind"] != "plain":
        g, u = v[:, :H], v[:, H:]
        if c["kind"] == "swiglu":
            v = _silu(g) * u
        else:
            d, p = s["d"].float(), torch.sigmoid(g)
            v = torch.cat([d * u * (p * (1 + g * (1 - p))), d * (g * p)], 1)
    out = {}
    if c["rows"]:
        out["codes"], out["sf"] = _scaled(v, (1, 128))
    if c["cols"]:
        out["col_codes"], out["col_sf"] = _scaled(v, (128, 1))
    return out


def _best(v, k):
    """Indices of the k largest, ties to the lowest; -1 where only -inf is left."""
    val, idx = torch.sort(v, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    return torch.where(val > -math.inf, idx, torch.full_like(idx, -1))


def _choose(c, L, bias):
    """The k largest keys of the best groups.  Keys are 32-bit sums, the sigmoid among them rounded from 64 bits, because
    which of two close ones is larger decides an index."""
    T, E, G = c["T"], c["E"], c["groups"]
    key = L
    if c["score"] == "sigmoid":
        key = torch.where(L > -math.inf, torch.sigmoid(L.double()).float(), L)
    if bias is not None:
        key = key + bias
    top = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
    rank = top[:, :, 0]
    if c["group_score"] == "top2" and E // G > 1:
        second = top[:, :, 1]
        rank = rank + torch.where(second > -math.inf, second, torch.zeros_like(second))
    at = _best(rank, c["topk_groups"])
    use = torch.zeros(T, G + 1, dtype=torch.bool, device=L.device).scatter_(1, torch.where(at >= 0, at, torch.full_like(at, G)), True)
    use = use[:, :G].repeat_interleave(E // G, 1)
    return _best(torch.where(use, key, torch.full_like(key, -math.inf)), c["k"])


def _scores(c, L):
    if c["score"] == "sigmoid":
        return torch.sigmoid(L)
    m = L.amax(1, keepdim=True)
    e = torch.exp(L - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    L = s["logits"].float()
    idx = _choose(c, L, s["bias"])
    on = idx >= 0
    p = _scores(c, L)
    w = torch.where(on, torch.gather(p, 1, idx.clamp(min=0)), torch.zeros_like(p[:, :1]))
    w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    out = {"topk_idx": idx.to(torch.int32), "topk_weights": w}
    if not c["train"]:
        return out
    real = (L > -math.inf).any(1)
    slot = torch.where(on, idx, torch.full_like(idx, E))
    picked = torch.zeros(T, E + 1, device=L.device).scatter_(1, slot, 1.0)[:, :E]
    at = torch.arange(T, device=L.device)
    off = s["seq_offsets"] if s["seq_offsets"] is not None else torch.tensor([0, T], device=L.device)
    seq = ((at[None] >= off[:-1, None]) & (at[None] < off[1:, None]) & real[None]).float()
    n = seq.sum(1)
    q = p if c["score"] == "softmax" else p / p.sum(1, keepdim=True).clamp(min=1e-30)
    counts, mean = seq @ picked, (seq @ q) / n.clamp(min=1)[:, None]
    f = E * counts / (k * n.clamp(min=1)[:, None])
    seqs = (n > 0).sum().clamp(min=1).float()
    loss = BALANCE_COEF * (f * mean).sum() / seqs
    C = seq.t() @ (BALANCE_COEF * f / (seqs * n.clamp(min=1)[:, None]))
    d = q * (C - (q * C).sum(1, keepdim=True))
    slope = 1 - p if c["score"] == "sigmoid" else torch.ones_like(p)
    g = torch.zeros(T, E + 1, device=L.device).scatter_(1, slot, s["d_weights"])[:, :E]
    W = torch.zeros(T, E + 1, device=L.device).scatter_(1, slot, w)[:, :E]
    d = slope * (d * s["d_loss"] + W * (g - (W * g).sum(1, keepdim=True)))
    out.update(loss=torch.stack([loss, loss, torch.zeros_like(loss)]), counts=counts.round().to(torch.int32), prob_mean=mean,
               seq_tokens=n.round().to(torch.int32), d_logits=d.to(s["logits"].dtype))
    return out


# ---- the calls -------------------------------------------------------------
def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn)


def _own_linear(s):
    o = s["op"].forward(s["x"], s["x_sf"], s["w"], s["w_sf"], add=s["add"], out=s["out"])
    return {"codes": _e4m3(o.codes), "sf": o.sf} if s["case"]["quant"] else {"y": o}


def _own_grad(s):
    if s["case"]["of"] == "input":
        return {"dinput": s["op"].backward_input(s["dy"], s["dy_sf"], s["w"], s["w_sf"], add=s["add"], out=s["out"])}
    return {"dweight": s["op"].backward_weight(s["dy"], s["dy_sf"], s["x"], s["x_sf"], add=s["add"], out=s["out"])}


def _own_quant(s):
    c, op = s["case"], s["op"]
    if c["kind"] == "blocks":
        o = op.weights(s["v"], out=s["out"])
    elif c["kind"] == "swiglu_grad":
        o = op.backward(s["d"], s["v"], out=s["out"])
    else:
        o = op.forward(s["v"], out=s["out"])
    out = {}
    if c["rows"]:
        out["codes"], out["sf"] = _e4m3(o.codes), o.sf
    if c["cols"]:
        out["col_codes"], out["col_sf"] = _e4m3(o.col_codes), o.col_sf
    return out


def _own_route(s):
    c, op = s["case"], s["op"]
    if not c["train"]:
        o = op.forward(s["logits"], s["bias"], out=s["out"])
        return {"topk_idx": o.topk_idx, "topk_weights": o.topk_weights}
    o = op.forward_train(s["logits"], s["bias"], s["seq_offsets"], out=s["out"])
    d = op.backward(s["logits"], o, d_weights=s["d_weights"], d_loss=s["d_loss"], out=s["d_logits"])
    return {"topk_idx": o.topk_idx, "topk_weights": o.topk_weights, "loss": o.loss, "counts": o.counts, "prob_mean": o.prob_mean,
            "seq_tokens": o.seq_tokens, "d_logits": d}


def run(state):
    forms = {"route": (_plain_route, _own_route), "linear": (_plain_linear, _own_linear), "grad": (_plain_grad, _own_grad),
             "quant": (_plain_quant, _own_quant)}
    return forms[state["case"]["op"]][own](state)


# ---- work ------------------------------------------------------------------
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        E, k, S, es = c["E"], c["k"], c["S"], SIZE[c["logits"]]
        fwd = T * E * es + 8 * T * k + (4 * E if c["bias"] else 0)
        if not c["train"]:
            return {"bytes": fwd, "flops": T * (6 * E + 4 * k)}
        return {"bytes": fwd + T * E * es + 4 * T * k + 8 * S * E + 8 * S + 16, "flops": T * (16 * E + 8 * k)}
    if c["op"] == "quant":
        H, es = c["H"], SIZE[c["dtype"]]
        if c["kind"] == "blocks":
            return {"bytes": T * H * (es + 1) + 4 * _up(T) * _up(H), "flops": 3 * T * H}
        wide = H * (2 if c["kind"] == "swiglu_grad" else 1)
        read = T * H * es * {"plain": 1, "swiglu": 2, "swiglu_grad": 3}[c["kind"]]
        wrote = c["rows"] * (T * wide + 4 * T * _up(wide)) + c["cols"] * (T * wide + 4 * _up(T) * wide)
        return {"bytes": read + wrote, "flops": T * wide * ({"plain": 0, "swiglu": 5, "swiglu_grad": 6}[c["kind"]] + 3)}
    N, K, size = c["N"], c["K"], SIZE[c["out"]]
    flops = 2 * T * N * K
    if c["op"] == "linear":
        n_out = N // 2 if c["act"] == "swiglu" else N
        out = T * n_out + 4 * T * _up(n_out) if c["quant"] else T * n_out * size * (1 + c["add"])
        return {"bytes": T * K + 4 * T * _up(K) + N * K + 4 * _up(N) * _up(K) + out, "flops": flops}
    if c["of"] == "input":
        return {"bytes": T * N + 4 * T * _up(N) + N * K + 4 * _up(N) * _up(K) + T * K * size * (1 + c["add"]), "flops": flops}
    return {"bytes": T * (N + K) + 4 * _up(T) * (N + K) + N * K * size * (1 + c["add"]), "flops": flops}


# ---- exact values ----------------------------------------------------------
def _value(codes, sf, axis):
    """The numbers that E4M3 codes stand for, from their bits, in 64 bits; axis: along which a scale covers 128 (2: both)."""
    b = codes.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    v = torch.where(b > 127, -v, v)
    row, col = (torch.arange(n, device=v.device) for n in v.shape)
    return v * sf.double()[row // 128 if axis != 1 else row][:, col // 128 if axis != 0 else col]


def _to_grid(v):
    """Nearest E4M3 value, ties to even, by arithmetic on the exponent: 3 fraction bits, smallest step 2^-9, largest 448."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 4).clamp(min=-9))
    return torch.sign(v) * torch.round(a / step) * step


def _exact_scaled(v, along):
    """Codes' values and scales along axis `along` (2: blocks of both)."""
    R, C = v.shape
    codes = torch.empty_like(v)
    if along == 2:
        sf = torch.zeros(_up(R), _up(C), dtype=torch.float64, device=v.device)
        for i in range(sf.shape[0]):
            for j in range(sf.shape[1]):
                b = v[128 * i:128 * i + 128, 128 * j:128 * j + 128]
                sf[i, j] = b.abs().max() / 448
                codes[128 * i:128 * i + 128, 128 * j:128 * j + 128] = _to_grid(b / sf[i, j]) if sf[i, j] > 0 else 0
        return codes, sf
    sfs = []
    for i, b in enumerate(torch.split(v, 128, along)):
        sf = b.abs().max(along, keepdim=True).values / 448
        q = torch.where(sf > 0, _to_grid(b / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(b))
        (codes[128 * i:128 * i + 128] if along == 0 else codes[:, 128 * i:128 * i + 128]).copy_(q)
        sfs.append(sf)
    return codes, torch.cat(sfs, along)


def _exact_linear(c, d):
    y = torch.einsum("tk,nk->tn", _value(d["x"], d["x_sf"], 1), _value(d["w"], d["w_sf"], 2))
    if c["act"] == "swiglu":
        g, u = torch.chunk(y, 2, 1)
        y = g / (1 + torch.exp(-g)) * u
    if c["quant"]:
        q, sf = _exact_scaled(y, 1)
        return {"codes": q, "sf": sf}
    return {"y": y if d["add"] is None else y + d["add"].double()}


def _exact_grad(c, d):
    if c["of"] == "input":
        r = torch.einsum("tn,nk->tk", _value(d["dy"], d["dy_sf"], 1), _value(d["w"], d["w_sf"], 2))
    else:
        r = torch.einsum("tn,tk->nk", _value(d["dy"], d["dy_sf"], 0), _value(d["x"], d["x_sf"], 0))
    return {"d" + c["of"]: r if d["add"] is None else r + d["add"].double()}


def _exact_quant(c, d):
    v = d["v"].double()
    if c["kind"] == "blocks":
        q, sf = _exact_scaled(v, 2)
        return {"codes": q, "sf": sf}
    if c["kind"] != "plain":
        g, u = torch.chunk(v, 2, 1)
        t = torch.exp(-g.abs())
        p = torch.where(g >= 0, 1 / (1 + t), t / (1 + t))
        if c["kind"] == "swiglu":
            v = g * p * u
        else:
            w = d["d"].double()
            v = torch.cat([w * u * (p + g * p * (1 - p)), w * g * p], 1)
    out = {}
    if c["rows"]:
        out["codes"], out["sf"] = _exact_scaled(v, 1)
    if c["cols"]:
        out["col_codes"], out["col_sf"] = _exact_scaled(v, 0)
    return out


def _exact_route(c, d):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = d["logits"].double()
    # the choice is made on 32-bit keys, so it is taken from them: the k largest by (key, -index) of the groups by (score, -index)
    key = x.float()
    if c["score"] == "sigmoid":
        key = torch.special.expit(x).float().masked_fill(x == -math.inf, -math.inf)
    if d["bias"] is not None:
        key = key + d["bias"]
    size = E // G
    two = torch.topk(key.reshape(T, G, size), min(2, size), dim=2).values
    if c["group_score"] == "max" or size == 1:
        mark = two[:, :, 0]
    else:
        mark = two[:, :, 0] + two[:, :, 1].masked_fill(two[:, :, 1] == -math.inf, 0.0)
    ahead = (mark.unsqueeze(1) > mark.unsqueeze(2)) | ((mark.unsqueeze(1) == mark.unsqueeze(2))
                                                       & (torch.arange(G, device=x.device) < torch.arange(G, device=x.device)[:, None]))
    best = ahead.sum(2) < c["topk_groups"]
    key = key.masked_fill(~best.repeat_interleave(size, 1), -math.inf)
    order = torch.argsort(-key, dim=1, stable=True)[:, :k]
    idx = order.masked_fill(torch.gather(key, 1, order) == -math.inf, -1)
    valid = (x > -math.inf).any(1)
    safe = torch.where(valid.unsqueeze(1), x, torch.zeros_like(x))
    if c["score"] == "softmax":
        raw = torch.exp(safe - torch.logsumexp(safe, 1).unsqueeze(1)) * valid.unsqueeze(1)
        share, slope = raw, torch.ones_like(raw)
    else:
        raw = torch.special.expit(x)
        share, slope = raw / raw.sum(1, keepdim=True).clamp(min=1e-300), 1 - raw
    hit = torch.zeros(T, E + 1, dtype=torch.float64, device=x.device)
    hit.scatter_(1, idx.masked_fill(idx < 0, E), 1.0)
    hit = hit[:, :E]
    top = raw * hit / (raw * hit).sum(1, keepdim=True).clamp(min=1e-300)
    out = {"topk_idx": None, "topk_weights": torch.gather(top, 1, idx.clamp(min=0)) * (idx >= 0)}
    if not c["train"]:
        return out
    off = d["seq_offsets"].tolist() if d["seq_offsets"] is not None else [0, T]
    spans = list(zip(off[:-1], off[1:]))
    n = [int(valid[a:b].sum()) for a, b in spans]
    used = max(1, sum(v > 0 for v in n))
    mean = torch.zeros(len(n), E, dtype=torch.float64, device=x.device)
    total, g = torch.zeros((), dtype=torch.float64, device=x.device), torch.zeros_like(x)
    for i, (a, b) in enumerate(spans):
        if n[i] == 0:
            continue
        on = valid[a:b].unsqueeze(1)
        mean[i] = (share[a:b] * on).sum(0) / n[i]
        load = (hit[a:b] * on).sum(0) * (E / (k * n[i]))
        total = total + BALANCE_COEF * (load * mean[i]).sum() / used
        pull = load * (BALANCE_COEF / used / n[i])
        g[a:b] += share[a:b] * slope[a:b] * (pull - (share[a:b] * pull).sum(1, keepdim=True)) * on
    g = g * d["d_loss"].double()
    W = torch.zeros(T, E + 1, dtype=torch.float64, device=x.device)
    W.scatter_add_(1, idx.masked_fill(idx < 0, E), d["d_weights"].double())
    W = W[:, :E]
    g = g + top * slope * (W - (top * W).sum(1, keepdim=True))
    out.update(loss=torch.stack([total, total, torch.zeros_like(total)]), counts=None, prob_mean=mean, seq_tokens=None, d_logits=g)
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    return {"route": _exact_route, "linear": _exact_linear, "grad": _exact_grad, "quant": _exact_quant}[case["op"]](case, d)
