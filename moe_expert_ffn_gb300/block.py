"""The MoE block around the expert layer: BlockNorm, Router and Fp4Linear.

Like MoELayer these allocate device memory through PyTorch and turn error
codes into exceptions; shapes, types, devices and pitches are checked, and
pointers marshalled, in _bind (csrc/bind.cpp); everything they compute runs in
the CUDA library (include/moe.h).  Every call takes ``out`` buffers made once
with ``buffers()`` / ``grad_buffers()``, so that a decode loop allocates
nothing, and allocates them itself, as memory of the stream it runs on, when
it gets none.

They take no part in autograd: outputs have no graph, gradients come from the
backward() calls, and a forward call whose inputs require gradients (outside
torch.no_grad()) warns of that.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import MOE_ERR_INVALID_ARG, Fp4LinearConfig, MoEError, NormConfig, RouterConfig, _check, lib

DTYPES = {torch.bfloat16: 0, torch.float32: 1}
GATES = {None: 0, "channel": 1, "token": 2}
QUANTS = {None: 0, "fp8": 1, "ue8m0": 2}
SCORES = {"softmax": 0, "sigmoid": 1}
BIASES = {"logit": 0, "score": 1}
ACTS = {None: 0, "swiglu": 1}
FP4_LINEAR_MAX_TOKENS = 16


def _device(device):
    d = torch.device(device if device is not None else "cuda")
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


def _choice(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {list(table)}, got {key!r}")
    return table[key]


try:   # the stream's handle without building a Stream object
    from torch._C import _cuda_getCurrentRawStream as _current_stream
except ImportError:   # pragma: no cover
    def _current_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _stream(stream, index):
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(index) if index >= 0 else 0


def _index(device):
    """What Tensor.get_device() gives on `device` (-1: not a GPU)."""
    return device.index if device.type == "cuda" else -1


def _bind():
    """The module that takes tensors to the library (raises if it was not built)."""
    try:
        from . import _bind as b
    except ImportError as e:
        raise RuntimeError("moe_expert_ffn_gb300/_bind.so is missing or was built against another PyTorch: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`") from e
    if b.torch_version != torch.__version__.split("+")[0]:
        raise RuntimeError(f"moe_expert_ffn_gb300/_bind.so was built against PyTorch {b.torch_version}: build it again")
    return b


def _made(stream, make, *args):
    """What a call allocates itself: memory of the stream it runs on, so that it goes back to that one."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _address(fn):
    return ctypes.cast(fn, ctypes.c_void_p).value


class NormOutput:
    """What BlockNorm.forward writes: h, n, codes, sf, rstd_post, rstd_pre (None where absent)."""
    __slots__ = ("h", "n", "codes", "sf", "rstd_post", "rstd_pre")


class NormGrads:
    """What BlockNorm.backward writes: dresidual, dy, dw_post, dgate, dw_pre (None where absent), and the workspace of
    partial sums that it writes on the way (None or unset: every call allocates one)."""
    __slots__ = ("dresidual", "dy", "dw_post", "dgate", "dw_pre", "workspace")


class BlockNorm:
    """The norms after one block and before the next in one pass:
    h = residual_scale * residual + gate * rmsnorm(y) * w_post, then n = rmsnorm(h) * w_pre,
    with n also as the expert layer's quantised input (``quant``: "fp8" = E4M3 with f32 scales per 128
    columns, "ue8m0" = E4M3 with UE8M0 scales per 32).  ``gate`` is None, "channel" ([hidden]) or
    "token" ([T]).  y is optional in forward (the first norm of a network), w_post and w_pre too."""

    def __init__(self, hidden, eps=1e-6, residual_scale=1.0, gate=None, quant=None, dtype=torch.bfloat16,
                 param_dtype=torch.float32, device=None):
        self.hidden, self.dtype, self.param_dtype, self.gate, self.quant = int(hidden), dtype, param_dtype, gate, quant
        self.device = _device(device)
        self.cfg = NormConfig(int(hidden), _choice(DTYPES, dtype, "dtype"), _choice(DTYPES, param_dtype, "param_dtype"),
                              _choice(GATES, gate, "gate"), _choice(QUANTS, quant, "quant"), float(eps), float(residual_scale))
        if lib().moe_norm_workspace_bytes(self.cfg, 1) == 0:
            raise MoEError(MOE_ERR_INVALID_ARG, "norm config")
        self._dev, b = _index(self.device), _bind()
        self._cfg, self._fwd, self._bwd = ctypes.addressof(self.cfg), b.norm_forward, b.norm_backward
        self._fwd_at, self._bwd_at = _address(lib().moe_norm_forward), _address(lib().moe_norm_backward)
        self._ws_at = _address(lib().moe_norm_workspace_bytes)

    def buffers(self, num_tokens, block=True, post=True, pre=True, normed=True) -> NormOutput:
        """Outputs of a forward of `num_tokens`: with y (`block`), w_post (`post`), w_pre (`pre`), n (`normed`)."""
        T, H, dev = num_tokens, self.hidden, self.device
        o = NormOutput()
        o.h = torch.empty(T, H, dtype=self.dtype, device=dev) if block else None
        o.rstd_post = torch.empty(T, dtype=torch.float32, device=dev) if block and post else None
        o.rstd_pre = torch.empty(T, dtype=torch.float32, device=dev) if pre else None
        o.n = torch.empty(T, H, dtype=self.dtype, device=dev) if pre and (normed or not self.quant) else None
        o.codes = o.sf = None
        if pre and self.quant:
            o.codes = torch.empty(T, H, dtype=torch.uint8, device=dev)
            o.sf = (torch.empty(T, H // 128, dtype=torch.float32, device=dev) if self.quant == "fp8"
                    else torch.empty(T, H // 32, dtype=torch.uint8, device=dev))
        return o

    def _workspace(self, num_tokens):
        return torch.empty(lib().moe_norm_workspace_bytes(self.cfg, num_tokens), dtype=torch.uint8, device=self.device)

    def grad_buffers(self, num_tokens, block=True, post=True, pre=True) -> NormGrads:
        """Outputs and workspace of a backward pass of `num_tokens`; passes with buffers of their own may run concurrently."""
        T, H, dev = num_tokens, self.hidden, self.device
        g = NormGrads()
        g.dresidual = torch.empty(T, H, dtype=self.dtype, device=dev)
        g.dy = torch.empty(T, H, dtype=self.dtype, device=dev) if block else None
        g.dw_post = torch.empty(H, dtype=torch.float32, device=dev) if block and post else None
        g.dw_pre = torch.empty(H, dtype=torch.float32, device=dev) if pre else None
        g.dgate = (torch.empty(H if self.gate == "channel" else T, dtype=torch.float32, device=dev)
                   if block and self.gate else None)
        g.workspace = self._workspace(T)
        return g

    def forward(self, residual, y=None, w_post=None, gate=None, w_pre=None, normed=True, out=None, stream=None) -> NormOutput:
        if out is None:
            out = _made(stream, self.buffers, residual.shape[0], y is not None, w_post is not None, w_pre is not None, normed)
        rc = self._fwd(self._fwd_at, self._cfg, self._dev, _stream(stream, self._dev),
                       residual, y, w_post, gate, w_pre, out.h, out.n, out.codes, out.sf, out.rstd_post, out.rstd_pre)
        if rc:
            _check(rc, "moe_norm_forward")
        return out

    def backward(self, h, dh=None, dn=None, y=None, w_post=None, gate=None, w_pre=None, rstd_post=None, rstd_pre=None,
                 out=None, stream=None) -> NormGrads:
        """Gradients from dh (of the stream h) and dn (of the normed n)."""
        T = h.shape[0]
        if out is None:
            out = _made(stream, self.grad_buffers, T, y is not None, w_post is not None, w_pre is not None)
        ws = getattr(out, "workspace", None)
        if ws is None:
            ws = _made(stream, self._workspace, T)
        rc = self._bwd(self._bwd_at, self._cfg, self._dev, _stream(stream, self._dev), h, dh, dn, y, w_post, gate, w_pre,
                       rstd_post, rstd_pre, out.dresidual, out.dy, out.dw_post, out.dgate, out.dw_pre, ws, self._ws_at)
        if rc:
            _check(rc, "moe_norm_backward")
        return out


class RouterOutput:
    """What Router writes: topk_idx, topk_weights and, with the losses, loss ([3]: total, balance, z),
    counts [S, E], prob_mean [S, E], seq_tokens [S] (views of ``tokens`` [S + 2]) and the seq_offsets they go by."""
    __slots__ = ("topk_idx", "topk_weights", "loss", "counts", "prob_mean", "seq_tokens", "tokens", "seq_offsets")


class Router:
    """Top-k router: topk_idx and topk_weights for MoELayer.forward from logits, the balance and z losses
    with per-sequence expert counts, and the gradient of the logits.  A bias, which takes part in the choice alone, is
    added to the logits or (``bias_on`` "score", with sigmoid scores) to the scores.  Losses use a workspace of this
    object: two loss calls of one Router must not run concurrently."""

    def __init__(self, num_experts, topk, score="softmax", renormalize=True, weight_scale=1.0, balance_coef=0.0, z_coef=0.0,
                 logits_dtype=torch.float32, max_tokens=None, max_seqs=1, device=None, bias_on="logit"):
        self.num_experts, self.topk, self.logits_dtype = int(num_experts), int(topk), logits_dtype
        self.max_tokens, self.max_seqs = max_tokens, int(max_seqs)
        self.device = _device(device)
        self.cfg = RouterConfig(int(num_experts), int(topk), _choice(SCORES, score, "score"), int(bool(renormalize)),
                                _choice(DTYPES, logits_dtype, "logits_dtype"), float(weight_scale), float(balance_coef),
                                float(z_coef), _choice(BIASES, bias_on, "bias_on"))
        need = lib().moe_router_workspace_bytes(self.cfg, 0 if max_tokens is None else int(max_tokens), self.max_seqs)
        if need == 0:
            raise MoEError(MOE_ERR_INVALID_ARG, "router config")
        self._dev, self._cfg, L, b = _index(self.device), ctypes.addressof(self.cfg), lib(), _bind()
        self._fwd, self._bal, self._bwd = b.router_forward, b.balance_loss, b.router_backward
        self._fwd_at, self._bal_at, self._bwd_at = (_address(L.moe_router_forward), _address(L.moe_balance_loss),
                                                    _address(L.moe_router_backward))
        # only the loss calls need it: they need to know max_tokens
        self._workspace = None if max_tokens is None else torch.empty(need, dtype=torch.uint8, device=self.device)
        self._limits = (-1 if max_tokens is None else int(max_tokens), self.max_seqs,
                        None if max_tokens is None else self._workspace.data_ptr())

    def buffers(self, num_tokens, num_seqs=None, choice=True) -> RouterOutput:
        """Outputs of a call on `num_tokens`, with those of the losses for `num_seqs` sequences, and without those of the
        choice where it is made elsewhere."""
        T, k, E, dev = num_tokens, self.topk, self.num_experts, self.device
        o = RouterOutput()
        o.topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev) if choice else None
        o.topk_weights = torch.empty(T, k, dtype=torch.float32, device=dev) if choice else None
        o.loss = o.counts = o.prob_mean = o.seq_tokens = o.tokens = o.seq_offsets = None
        if num_seqs is not None:
            o.loss = torch.empty(3, dtype=torch.float32, device=dev)
            o.counts = torch.empty(num_seqs, E, dtype=torch.int32, device=dev)
            o.prob_mean = torch.empty(num_seqs, E, dtype=torch.float32, device=dev)
            o.tokens = torch.empty(num_seqs + 2, dtype=torch.int32, device=dev)
            o.seq_tokens = o.tokens[:num_seqs]
        return o

    def _grad_buffer(self, num_tokens):
        return torch.empty(num_tokens, self.num_experts, dtype=self.logits_dtype, device=self.device)

    def forward(self, logits, bias=None, out=None, stream=None) -> RouterOutput:
        """topk_idx and topk_weights of logits [T, E] (bias f32 [E]: for the choice alone)."""
        if out is None:
            out = _made(stream, self.buffers, logits.shape[0])
        rc = self._fwd(self._fwd_at, self._cfg, self._dev, _stream(stream, self._dev), logits, bias, out.topk_idx, out.topk_weights)
        if rc:
            _check(rc, "moe_router_forward")
        return out

    def forward_train(self, logits, bias=None, seq_offsets=None, out=None, stream=None) -> RouterOutput:
        """The same with the losses, in one pass; seq_offsets int32 [S + 1], or None for one sequence."""
        if out is None:
            out = _made(stream, self.buffers, logits.shape[0], 1 if seq_offsets is None else seq_offsets.shape[0] - 1)
        rc = self._fwd(self._fwd_at, self._cfg, self._dev, _stream(stream, self._dev), logits, bias, out.topk_idx, out.topk_weights,
                       seq_offsets, out.loss, out.counts, out.prob_mean, out.tokens, *self._limits)
        if rc:
            _check(rc, "moe_router_forward")
        out.seq_offsets = seq_offsets
        return out

    def balance_loss(self, logits, topk_idx, seq_offsets=None, out=None, stream=None) -> RouterOutput:
        """The losses of a choice made elsewhere.  The result has that choice as its topk_idx, for backward, and no
        weights; of `out` the loss tensors are used, and its own choice stays what it is."""
        if out is None:
            out = _made(stream, self.buffers, logits.shape[0], 1 if seq_offsets is None else seq_offsets.shape[0] - 1, False)
        rc = self._bal(self._bal_at, self._cfg, self._dev, _stream(stream, self._dev), logits, topk_idx,
                       seq_offsets, out.loss, out.counts, out.prob_mean, out.tokens, *self._limits)
        if rc:
            _check(rc, "moe_balance_loss")
        o = RouterOutput()
        o.topk_idx, o.topk_weights = topk_idx, None
        o.seq_offsets = out.seq_offsets = seq_offsets
        o.loss, o.counts, o.prob_mean, o.seq_tokens, o.tokens = out.loss, out.counts, out.prob_mean, out.seq_tokens, out.tokens
        return o

    def backward(self, logits, fwd, d_weights=None, d_loss=None, seq_offsets=None, out=None, stream=None):
        """d_logits through topk_weights (`d_weights` [T, k]) and through loss[0] (`d_loss`, an f32 scalar on the
        device); `fwd` is what the forward call returned, and seq_offsets need not be given again."""
        if out is None:
            out = _made(stream, self._grad_buffer, logits.shape[0])
        args = (self._bwd_at, self._cfg, self._dev, _stream(stream, self._dev), logits,
                fwd.topk_idx if d_weights is not None else None, d_weights, out)
        if d_loss is not None:
            if seq_offsets is None:
                seq_offsets = getattr(fwd, "seq_offsets", None)
            args += (d_loss, seq_offsets, fwd.loss, fwd.counts, fwd.prob_mean, fwd.tokens, *self._limits)
        rc = self._bwd(*args)
        if rc:
            _check(rc, "moe_router_backward")
        return out


class Fp4Linear:
    """y = act(x W^T) (+ add) of 1 to 16 tokens with E2M1 weights under UE8M0 scales per 32 (the layer's FP4
    format); act "swiglu": rows [0, N/2) gate, [N/2, N) up, N/2 outputs."""

    def __init__(self, in_features, out_features, act=None, out_dtype=torch.bfloat16, act_clamp=math.inf, device=None):
        self.device, self.out_dtype = _device(device), out_dtype
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.out_columns = self.out_features // 2 if act == "swiglu" else self.out_features
        self.cfg = Fp4LinearConfig(int(in_features), int(out_features), _choice(ACTS, act, "act"),
                                   _choice(DTYPES, out_dtype, "out_dtype"), float(act_clamp))
        need = lib().moe_fp4_linear_weight_bytes(self.cfg)
        if need == 0:
            raise MoEError(MOE_ERR_INVALID_ARG, "fp4 linear config")
        self.weights = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._cfg, self._ready, self._dev, b = ctypes.addressof(self.cfg), False, _index(self.device), _bind()
        self._fwd, self._fwd_at = b.linear_forward, _address(lib().moe_fp4_linear_forward)

    def transform_weights(self, w, w_sf, stream=None):
        _check(_bind().linear_transform(_address(lib().moe_fp4_linear_transform_weights), self._cfg, self._dev,
                                        _stream(stream, self._dev), w, w_sf, self.weights.data_ptr()), "moe_fp4_linear_transform_weights")
        self._ready = True

    def buffers(self, num_tokens):
        return torch.empty(num_tokens, self.out_columns, dtype=self.out_dtype, device=self.device)

    def forward(self, x, add=None, out=None, stream=None):
        if not self._ready:
            raise MoEError(-6, "moe_fp4_linear_forward")
        if out is None:
            out = _made(stream, self.buffers, x.shape[0])
        rc = self._fwd(self._fwd_at, self._cfg, self._dev, _stream(stream, self._dev), x, add, out, self.weights.data_ptr())
        if rc:
            _check(rc, "moe_fp4_linear_forward")
        return out
