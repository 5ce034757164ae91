"""The MoE block around the expert layer: BlockNorm, Router and Fp4Linear.

Like MoELayer these allocate device memory through PyTorch, check shapes and
types, marshal pointers and turn error codes into exceptions; everything they
compute runs in the CUDA library (include/moe.h).  Every call takes ``out``
buffers made once with ``buffers()`` / ``grad_buffers()``, so that a decode
loop allocates nothing, and allocates them itself when it gets none.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (MOE_ERR_INVALID_ARG, Fp4LinearConfig, MoEError, NormConfig, NormGradIO, NormIO, RouterConfig,
               BalanceIO, _check, lib)

DTYPES = {torch.bfloat16: 0, torch.float32: 1}
GATES = {None: 0, "channel": 1, "token": 2}
QUANTS = {None: 0, "fp8": 1, "ue8m0": 2}
SCORES = {"softmax": 0, "sigmoid": 1}
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
    return _current_stream(index) if stream is None else stream.cuda_stream


def _index(device):
    """What Tensor.get_device() gives on `device` (-1: not a GPU)."""
    return device.index if device.type == "cuda" else -1


def _refuse(t, name, dtype, shape, what):
    raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} {what}, got {t.dtype} {tuple(t.shape)} with "
                     f"strides {t.stride()} on {t.device}")


def _rows(t, name, dtype, shape, index):
    """(pointer, row pitch) of a [rows, cols] tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(t, name, dtype, shape, "on the operator's device")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    pitch, step = t.stride()
    if (step != 1 and shape[1] > 1) or (shape[0] > 1 and pitch < shape[1]):
        _refuse(t, name, dtype, shape, "with contiguous rows that do not overlap")
    return t.data_ptr(), pitch if shape[0] > 1 else shape[1]


def _flat(t, name, dtype, shape, index):
    """Pointer of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, dtype, shape, "contiguous on the operator's device")
    return t.data_ptr()


class _Outputs:
    """Output tensors of a call and, once checked against an operator, their native description: a later call with the
    same ones only asks them for their addresses.  Replacing a tensor has it checked again."""
    __slots__ = ("_of", "_key", "_io", "_own")

    def __init__(self):
        for n in type(self).__slots__:
            object.__setattr__(self, n, None)
        object.__setattr__(self, "_of", None)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_of", None)

    def _bind(self, op, key, io, own):
        """Checked for calls of `op` described by `key`; `own`: (tensor, field of io) pairs."""
        for n, v in (("_io", io), ("_own", own), ("_key", key), ("_of", op)):
            object.__setattr__(self, n, v)


class NormOutput(_Outputs):
    """What BlockNorm.forward writes: h, n, codes, sf, rstd_post, rstd_pre (None where absent)."""
    __slots__ = ("h", "n", "codes", "sf", "rstd_post", "rstd_pre")


class NormGrads(_Outputs):
    """What BlockNorm.backward writes: dresidual, dy, dw_post, dgate, dw_pre (None where absent)."""
    __slots__ = ("dresidual", "dy", "dw_post", "dgate", "dw_pre")


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
        self._workspace, self._dev, self._width, self._channel = None, _index(self.device), (int(hidden),), gate == "channel"
        self._cfg = ctypes.byref(self.cfg)
        self._fwd, self._bwd, self._ws_bytes = lib().moe_norm_forward, lib().moe_norm_backward, lib().moe_norm_workspace_bytes

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

    def grad_buffers(self, num_tokens, block=True, post=True, pre=True) -> NormGrads:
        T, H, dev = num_tokens, self.hidden, self.device
        g = NormGrads()
        g.dresidual = torch.empty(T, H, dtype=self.dtype, device=dev)
        g.dy = torch.empty(T, H, dtype=self.dtype, device=dev) if block else None
        g.dw_post = torch.empty(H, dtype=torch.float32, device=dev) if block and post else None
        g.dw_pre = torch.empty(H, dtype=torch.float32, device=dev) if pre else None
        g.dgate = (torch.empty(H if self.gate == "channel" else T, dtype=torch.float32, device=dev)
                   if block and self.gate else None)
        return g

    def _params(self, io, T, w_post, gate, w_pre):
        dt, dev, width = self.param_dtype, self._dev, self._width
        io.w_post = None if w_post is None else _flat(w_post, "w_post", dt, width, dev)
        io.gate = None if gate is None else _flat(gate, "gate", dt, width if self._channel else (T,), dev)
        io.w_pre = None if w_pre is None else _flat(w_pre, "w_pre", dt, width, dev)

    @staticmethod
    def _check_all(io, wanted, index):
        """Checks (name, tensor, dtype, shape, pitched) outputs and writes them into io."""
        own = []
        for name, t, dtype, shape, pitched in wanted:
            if t is None:
                continue
            if pitched:
                ptr, pitch = _rows(t, name, dtype, shape, index)
                setattr(io, "ld_" + name, pitch)
            else:
                ptr = _flat(t, name, dtype, shape, index)
            setattr(io, name, ptr)
            own.append((t, name))
        return own

    def forward(self, residual, y=None, w_post=None, gate=None, w_pre=None, normed=True, out=None, stream=None) -> NormOutput:
        T, H, dt, dev = residual.shape[0], self.hidden, self.dtype, self._dev
        if out is None:
            out = self.buffers(T, y is not None, w_post is not None, w_pre is not None, normed)
        key = (T, y is None, w_post is None, w_pre is None)
        if out._of is self and out._key == key:
            io = out._io
            for t, name in out._own:
                setattr(io, name, t.data_ptr())
        else:
            f32, u8, shape, block, pre = torch.float32, torch.uint8, (T, H), y is not None, w_pre is not None
            io = NormIO()
            quant = pre and self.quant
            if block and out.h is None or quant and (out.codes is None or out.sf is None):
                raise ValueError("out lacks h, codes or sf")
            own = self._check_all(io, (
                ("h", out.h if block else None, dt, shape, True), ("n", out.n if pre else None, dt, shape, True),
                ("codes", out.codes if quant else None, u8, shape, False),
                ("sf", out.sf if quant else None, f32 if self.quant == "fp8" else u8, (T, H // (128 if self.quant == "fp8" else 32)), False),
                ("rstd_post", out.rstd_post if block and w_post is not None else None, f32, (T,), False),
                ("rstd_pre", out.rstd_pre if pre else None, f32, (T,), False)), dev)
            out._bind(self, key, io, own)
        shape = (T, H)
        io.residual, io.ld_residual = _rows(residual, "residual", dt, shape, dev)
        if y is not None:
            io.y, io.ld_y = _rows(y, "y", dt, shape, dev)
        self._params(io, T, w_post, gate, w_pre)
        rc = self._fwd(self._cfg, T, io, _current_stream(dev) if stream is None else stream.cuda_stream)
        if rc:
            _check(rc, "moe_norm_forward")
        return out

    def backward(self, h, dh=None, dn=None, y=None, w_post=None, gate=None, w_pre=None, rstd_post=None, rstd_pre=None,
                 out=None, stream=None) -> NormGrads:
        """Gradients from dh (of the stream h) and dn (of the normed n).  Uses a workspace of this object,
        so backward passes of one BlockNorm must not run concurrently."""
        T, H, dt, dev, f32 = h.shape[0], self.hidden, self.dtype, self._dev, torch.float32
        if out is None:
            out = self.grad_buffers(T, y is not None, w_post is not None, w_pre is not None)
        key = (T, y is None, w_post is None, w_pre is None, gate is None)
        shape = (T, H)
        if out._of is self and out._key == key:
            io = out._io
            for t, name in out._own:
                setattr(io, name, t.data_ptr())
        else:
            io = NormGradIO()
            wanted = (("dresidual", out.dresidual, dt, shape, True), ("dy", out.dy if y is not None else None, dt, shape, True),
                      ("dw_post", out.dw_post if w_post is not None else None, f32, self._width, False),
                      ("dw_pre", out.dw_pre if w_pre is not None else None, f32, self._width, False),
                      ("dgate", out.dgate if gate is not None else None, f32, self._width if self.gate == "channel" else (T,), False))
            out._bind(self, key, io, self._check_all(io, wanted, dev))
        io.h, io.ld_h = _rows(h, "h", dt, shape, dev)
        self._params(io, T, w_post, gate, w_pre)
        io.dh, io.ld_dh = (None, 0) if dh is None else _rows(dh, "dh", dt, shape, dev)
        io.dn, io.ld_dn = (None, 0) if dn is None else _rows(dn, "dn", dt, shape, dev)
        if y is not None:
            io.y, io.ld_y = _rows(y, "y", dt, shape, dev)
        io.rstd_post = None if w_post is None or rstd_post is None else _flat(rstd_post, "rstd_post", f32, (T,), dev)
        io.rstd_pre = None if w_pre is None or rstd_pre is None else _flat(rstd_pre, "rstd_pre", f32, (T,), dev)
        need = self._ws_bytes(self._cfg, T)
        if self._workspace is None or self._workspace.numel() < need:
            self._workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        rc = self._bwd(self._cfg, T, io, self._workspace.data_ptr(), _stream(stream, dev))
        if rc:
            _check(rc, "moe_norm_backward")
        return out


class RouterOutput(_Outputs):
    """What Router writes: topk_idx, topk_weights and, with the losses, loss ([3]: total, balance, z),
    counts [S, E], prob_mean [S, E], seq_tokens [S] (views of ``tokens`` [S + 2])."""
    __slots__ = ("topk_idx", "topk_weights", "loss", "counts", "prob_mean", "seq_tokens", "tokens")


class Router:
    """Top-k router: topk_idx and topk_weights for MoELayer.forward from logits, the balance and z losses
    with per-sequence expert counts, and the gradient of the logits.  Losses use a workspace of this
    object: two loss calls of one Router must not run concurrently."""

    def __init__(self, num_experts, topk, score="softmax", renormalize=True, weight_scale=1.0, balance_coef=0.0, z_coef=0.0,
                 logits_dtype=torch.float32, max_tokens=None, max_seqs=1, device=None):
        self.num_experts, self.topk, self.logits_dtype = int(num_experts), int(topk), logits_dtype
        self.max_tokens, self.max_seqs = max_tokens, int(max_seqs)
        self.device = _device(device)
        self.cfg = RouterConfig(int(num_experts), int(topk), _choice(SCORES, score, "score"), int(bool(renormalize)),
                                _choice(DTYPES, logits_dtype, "logits_dtype"), float(weight_scale), float(balance_coef),
                                float(z_coef))
        need = lib().moe_router_workspace_bytes(self.cfg, 0 if max_tokens is None else int(max_tokens), self.max_seqs)
        if need == 0:
            raise MoEError(MOE_ERR_INVALID_ARG, "router config")
        self._dev, self._bias_shape = _index(self.device), (int(num_experts),)
        self._cfg = ctypes.byref(self.cfg)
        L = lib()
        self._fwd, self._bal, self._bwd = L.moe_router_forward, L.moe_balance_loss, L.moe_router_backward
        # only the loss calls need it: they need to know max_tokens
        self._workspace = None if max_tokens is None else torch.empty(need, dtype=torch.uint8, device=self.device)

    def buffers(self, num_tokens, num_seqs=None) -> RouterOutput:
        """Outputs of a call on `num_tokens`, with those of the losses for `num_seqs` sequences."""
        T, k, E, dev = num_tokens, self.topk, self.num_experts, self.device
        o = RouterOutput()
        o.topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        o.topk_weights = torch.empty(T, k, dtype=torch.float32, device=dev)
        o.loss = o.counts = o.prob_mean = o.seq_tokens = o.tokens = None
        if num_seqs is not None:
            o.loss = torch.empty(3, dtype=torch.float32, device=dev)
            o.counts = torch.empty(num_seqs, E, dtype=torch.int32, device=dev)
            o.prob_mean = torch.empty(num_seqs, E, dtype=torch.float32, device=dev)
            o.tokens = torch.empty(num_seqs + 2, dtype=torch.int32, device=dev)
            o.seq_tokens = o.tokens[:num_seqs]
        return o

    def _losses(self, T, seq_offsets, out, write=True):
        S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
        if write and (self.max_tokens is None or T > self.max_tokens or S > self.max_seqs):
            raise ValueError(f"{T} tokens in {S} sequences: the router was made for losses of "
                             f"{self.max_tokens} tokens in {self.max_seqs}")
        if out._of is self and out._key == S:
            io = out._io
            for t, name in out._own:
                setattr(io, name, t.data_ptr())
        else:
            E, dev, f32, i32 = self.num_experts, self._dev, torch.float32, torch.int32
            io = BalanceIO()
            io.num_seqs = S
            own = BlockNorm._check_all(io, (("loss", out.loss, f32, (3,), False), ("counts", out.counts, i32, (S, E), False),
                                            ("prob_mean", out.prob_mean, f32, (S, E), False),
                                            ("seq_tokens", out.tokens, i32, (S + 2,), False)), dev)
            if len(own) != 4:
                raise ValueError("out lacks the outputs of the losses")
            out._bind(self, S, io, own)
        io.seq_offsets = None if seq_offsets is None else _flat(seq_offsets, "seq_offsets", torch.int32, (S + 1,), self._dev)
        return io

    def _forward(self, logits, bias, loss_seqs, seq_offsets, out, stream):
        T, E, k, dev = logits.shape[0], self.num_experts, self.topk, self._dev
        if out is None:
            out = self.buffers(T, loss_seqs)
        ptr, ld = _rows(logits, "logits", self.logits_dtype, (T, E), dev)
        b = None if bias is None else _flat(bias, "bias", torch.float32, self._bias_shape, dev)
        idx = _flat(out.topk_idx, "topk_idx", torch.int32, (T, k), dev)
        wts = _flat(out.topk_weights, "topk_weights", torch.float32, (T, k), dev)
        io = ws = None
        if loss_seqs is not None:
            io, ws = self._losses(T, seq_offsets, out), self._workspace.data_ptr()
        rc = self._fwd(self._cfg, T, ptr, ld, b, idx, wts, io, ws, _stream(stream, dev))
        if rc:
            _check(rc, "moe_router_forward")
        return out

    def forward(self, logits, bias=None, out=None, stream=None) -> RouterOutput:
        """topk_idx and topk_weights of logits [T, E] (bias f32 [E]: for the choice alone)."""
        return self._forward(logits, bias, None, None, out, stream)

    def forward_train(self, logits, bias=None, seq_offsets=None, out=None, stream=None) -> RouterOutput:
        """The same with the losses, in one pass; seq_offsets int32 [S + 1], or None for one sequence."""
        S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
        return self._forward(logits, bias, S, seq_offsets, out, stream)

    def balance_loss(self, logits, topk_idx, seq_offsets=None, out=None, stream=None) -> RouterOutput:
        """The losses of a choice made elsewhere."""
        T, E, dev = logits.shape[0], self.num_experts, self._dev
        if out is None:
            out = self.buffers(T, 1 if seq_offsets is None else seq_offsets.shape[0] - 1)
        ptr, ld = _rows(logits, "logits", self.logits_dtype, (T, E), dev)
        idx = _flat(topk_idx, "topk_idx", torch.int32, (T, self.topk), dev)
        io = self._losses(T, seq_offsets, out)
        rc = self._bal(self._cfg, T, ptr, ld, idx, io, self._workspace.data_ptr(), _stream(stream, dev))
        if rc:
            _check(rc, "moe_balance_loss")
        return out

    def backward(self, logits, fwd, d_weights=None, d_loss=None, seq_offsets=None, out=None, stream=None):
        """d_logits through topk_weights (`d_weights` [T, k]) and through loss[0] (`d_loss`, an f32 scalar on the
        device); `fwd` is what the forward call returned."""
        T, E, k, dev = logits.shape[0], self.num_experts, self.topk, self._dev
        if out is None:
            out = torch.empty(T, E, dtype=self.logits_dtype, device=self.device)
        ptr, ld = _rows(logits, "logits", self.logits_dtype, (T, E), dev)
        dptr, dld = _rows(out, "d_logits", self.logits_dtype, (T, E), dev)
        idx = dw = io = dl = None
        if d_weights is not None:
            idx = _flat(fwd.topk_idx, "topk_idx", torch.int32, (T, k), dev)
            dw = _flat(d_weights, "d_weights", torch.float32, (T, k), dev)
        if d_loss is not None:
            if d_loss.numel() != 1:
                raise ValueError("d_loss must hold one value")
            io, dl = self._losses(T, seq_offsets, fwd, write=False), _flat(d_loss, "d_loss", torch.float32, d_loss.shape, dev)
        rc = self._bwd(self._cfg, T, ptr, ld, idx, dw, io, dl, dptr, dld, _stream(stream, dev))
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
        self._cfg, self._ready, self._dev, self._fwd = ctypes.byref(self.cfg), False, _index(self.device), lib().moe_fp4_linear_forward

    def transform_weights(self, w, w_sf, stream=None):
        N, K, dev = self.out_features, self.in_features, self._dev
        wp = _flat(w, "w", torch.uint8, (N, K // 2), dev)
        sp = _flat(w_sf, "w_sf", torch.uint8, (N, K // 32), dev)
        _check(lib().moe_fp4_linear_transform_weights(self.cfg, wp, sp, self.weights.data_ptr(), _stream(stream, dev)),
               "moe_fp4_linear_transform_weights")
        self._ready = True

    def buffers(self, num_tokens):
        return torch.empty(num_tokens, self.out_columns, dtype=self.out_dtype, device=self.device)

    def forward(self, x, add=None, out=None, stream=None):
        if not self._ready:
            raise MoEError(-6, "moe_fp4_linear_forward")
        T, n, dev = x.shape[0], self.out_columns, self._dev
        if out is None:
            out = self.buffers(T)
        xp, ldx = _rows(x, "x", torch.bfloat16, (T, self.in_features), dev)
        yp, ldy = _rows(out, "y", self.out_dtype, (T, n), dev)
        ap, lda = (None, 0) if add is None else _rows(add, "add", self.out_dtype, (T, n), dev)
        rc = self._fwd(self._cfg, T, xp, ldx, self.weights.data_ptr(), ap, lda, yp, ldy, _stream(stream, dev))
        if rc:
            _check(rc, "moe_fp4_linear_forward")
        return out
