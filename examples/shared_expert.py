"""The shared expert of an MoE block in FP8: serving any number of tokens, and
training.

    python examples/shared_expert.py [--hidden 1024 --inter 512 --tokens 300 --steps 5]

    y = W_down . swiglu(W_gate_up . x)  (+ the routed experts' output)

Weights are kept in f32 and quantised per 128 x 128 after every update.  A
product takes its input with scales along the contracted axis: per 1 x 128 of
a token forward and for the input's gradient, per 128 tokens of a column for
the weight's gradient.  The quantiser writes both forms in one pass, and no
operand is ever transposed in memory.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_ffn_gb300 as moe  # noqa: E402


class SharedExpert:
    """`w_gate_up` f32 [2 inter, hidden] (rows [0, inter) gate, then up) and `w_down` f32 [hidden, inter]."""

    def __init__(self, w_gate_up, w_down):
        dev = w_down.device
        self.H, self.I = w_down.shape
        self.w_gate_up, self.w_down = w_gate_up, w_down
        self.gate_up = moe.Fp8Linear(self.H, 2 * self.I, device=dev)                                   # training: gate and up themselves
        self.act = moe.Fp8Linear(self.H, 2 * self.I, act="swiglu", quant="fp8", device=dev)            # serving: the down product's input
        self.down = moe.Fp8Linear(self.I, self.H, device=dev)
        self.quant = moe.Fp8Quant(self.H, device=dev)
        self.quant_act = moe.Fp8Quant(self.I, act="swiglu", device=dev)
        self.store = (moe.Fp8Quant(self.H, dtype=torch.float32, device=dev), moe.Fp8Quant(self.I, dtype=torch.float32, device=dev))
        self.q_gate_up, self.q_down = self.store[0].weight_buffers(2 * self.I), self.store[1].weight_buffers(self.H)
        self.refresh()

    def refresh(self):
        """The weights' codes after an update."""
        self.store[0].weights(self.w_gate_up, out=self.q_gate_up)
        self.store[1].weights(self.w_down, out=self.q_down)

    def buffers(self, tokens):
        """What a serving step writes on the way."""
        return self.quant.buffers(tokens), self.act.buffers(tokens)

    def forward(self, x, add=None, out=None, buffers=None):
        """bf16 [T, hidden] of x bf16 [T, hidden]; `add` is added (it may be `out`)."""
        q, mid = buffers or self.buffers(x.shape[0])
        self.quant.forward(x, out=q)
        self.act.forward(q.codes, q.sf, self.q_gate_up.codes, self.q_gate_up.sf, out=mid)
        return self.down.forward(mid.codes, mid.sf, self.q_down.codes, self.q_down.sf, add=add, out=out)

    def forward_train(self, x):
        """(y, what backward needs)."""
        q = self.quant.forward(x, cols=True)
        v = self.gate_up.forward(q.codes, q.sf, self.q_gate_up.codes, self.q_gate_up.sf)
        mid = self.quant_act.forward(v, cols=True)
        return self.down.forward(mid.codes, mid.sf, self.q_down.codes, self.q_down.sf), (q, v, mid)

    def backward(self, dy, saved, grads=None):
        """(dx, (dw_gate_up, dw_down)) from dy bf16 [T, hidden]; `grads` of earlier micro-batches are added to in place."""
        q, v, mid = saved
        dw_gate_up, dw_down = grads or (None, None)
        dq = self.quant.forward(dy, cols=True)
        dw_down = self.down.backward_weight(dq.col_codes, dq.col_sf, mid.col_codes, mid.col_sf, add=dw_down, out=dw_down)
        d_mid = self.down.backward_input(dq.codes, dq.sf, self.q_down.codes, self.q_down.sf)
        dv = self.quant_act.backward(d_mid, v)
        dw_gate_up = self.gate_up.backward_weight(dv.col_codes, dv.col_sf, q.col_codes, q.col_sf, add=dw_gate_up, out=dw_gate_up)
        dx = self.gate_up.backward_input(dv.codes, dv.sf, self.q_gate_up.codes, self.q_gate_up.sf)
        return dx, (dw_gate_up, dw_down)

    def update(self, grads, lr):
        """A step of gradient descent."""
        self.w_gate_up.sub_(grads[0], alpha=lr)
        self.w_down.sub_(grads[1], alpha=lr)
        self.refresh()


def random_expert(hidden, inter, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return SharedExpert(rand(2 * inter, hidden) / hidden ** 0.5, rand(hidden, inter) / inter ** 0.5)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("hidden", 1024), ("inter", 512), ("tokens", 300), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    student, teacher = random_expert(a.hidden, a.inter), random_expert(a.hidden, a.inter, seed=1)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    goal = teacher.forward(x).float()
    for i in range(a.steps):
        y, saved = student.forward_train(x)
        off = y.float() - goal
        _, grads = student.backward((off / off.numel() ** 0.5).to(torch.bfloat16), saved)
        student.update(grads, lr=0.05)
        print(f"step {i}: mean square difference from the other expert {off.square().mean().item():.4f}")
    assert moe.lib().moe_fp8_linear_status() == moe.MOE_OK


if __name__ == "__main__":
    main()
