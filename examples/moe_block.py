"""An MoE block of a transformer from the library's operators: serving steps
and training of the router.

    python examples/moe_block.py [--hidden 7168 --inter 2048 --experts 256 --topk 8 --tokens 16]

A block takes the residual stream h and the previous block's output y:

    h, n, codes, sf = BlockNorm(h, y)                 gate, residual sum, both norms, quantised input of the experts
    idx, weights    = Router(n W_r^T)                 top-k choice of the experts
    out             = MoELayer(codes, sf, idx, weights)
    out            += W_down . swiglu(W_gate_up . n)  the shared expert: FP4 weights up to 16 tokens, FP8 above

and hands (h, out) to the next block.  Every buffer of a step is made once, so
a step allocates nothing and can be captured into a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_ffn_gb300 as moe  # noqa: E402
import moe_synth  # noqa: E402
from examples.shared_expert import SharedExpert  # noqa: E402


class MoEBlock:
    """One block for up to `tokens` tokens, with random weights; FP4 weights in the routed experts too."""

    def __init__(self, tokens, hidden, inter, experts, topk, seed=0, device="cuda", groups=None, topk_groups=None):
        dev = torch.device(device)
        wl = moe_synth.custom(tokens, hidden, inter, experts, topk, seed=seed, wfmt=moe.MOE_W_FP4_E2M1_UE8M0_32)
        g = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.T, self.H, self.E = tokens, hidden, experts
        self.norm = moe.BlockNorm(hidden, gate="channel", quant="ue8m0", device=dev)
        self.router = moe.Router(experts, topk, balance_coef=1e-2, z_coef=1e-4, max_tokens=tokens, device=dev, groups=groups,
                                 topk_groups=topk_groups)
        self.experts = moe.MoELayer(tokens, hidden, inter, experts, topk, wfmt=wl.wfmt, device=torch.device("cuda", torch.cuda.current_device()))
        self.experts.transform_weights(*moe_synth.make_weights(wl, device=dev))
        w_gate_up, w_down = rand(2 * inter, hidden) / hidden ** 0.5, rand(hidden, inter) / inter ** 0.5
        self.few = tokens <= moe.FP4_LINEAR_MAX_TOKENS
        if self.few:
            self.gate_up = moe.Fp4Linear(hidden, 2 * inter, act="swiglu", device=dev)
            self.down = moe.Fp4Linear(inter, hidden, device=dev)
            self.shared = {"gate_up": moe_synth.pack_e2m1_rows(w_gate_up), "down": moe_synth.pack_e2m1_rows(w_down)}
            self.gate_up.transform_weights(*self.shared["gate_up"])
            self.down.transform_weights(*self.shared["down"])
        else:
            self.shared = SharedExpert(w_gate_up, w_down)
        self.w_post, self.w_pre = 1 + 0.1 * rand(hidden), 1 + 0.1 * rand(hidden)
        self.gate = 0.5 + 0.1 * rand(hidden)
        self.w_router = rand(experts, hidden) / hidden ** 0.5
        # the buffers of a step
        self.normed = self.norm.buffers(tokens)
        self.routed = self.router.buffers(tokens, num_seqs=1)
        self.logits = torch.empty(tokens, experts, device=dev)
        self.n32 = torch.empty(tokens, hidden, device=dev)
        self.mid = self.gate_up.buffers(tokens) if self.few else self.shared.buffers(tokens)
        self.out = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=dev)

    def _route_input(self, h, y):
        """The stream after the previous block, its normed forms and the router's logits."""
        o = self.norm.forward(h, y, w_post=self.w_post, gate=self.gate, w_pre=self.w_pre, out=self.normed)
        self.n32.copy_(o.n)
        torch.mm(self.n32, self.w_router.t(), out=self.logits)
        return o

    def step(self, h, y):
        """(stream, block output) of the next block from those of the previous one."""
        o = self._route_input(h, y)
        r = self.router.forward(self.logits, out=self.routed)
        self.experts.forward(o.codes, o.sf, r.topk_idx, r.topk_weights, y=self.out)
        if self.few:
            self.gate_up.forward(o.n, out=self.mid)
            self.down.forward(self.mid, add=self.out, out=self.out)
        else:
            self.shared.forward(o.n, add=self.out, out=self.out, buffers=self.mid)
        return o.h, self.out

    def train_router(self, h, y, lr):
        """One step of gradient descent of the router's weights on its balance and z losses; returns them and the
        largest expert's share of the tokens."""
        self._route_input(h, y)
        r = self.router.forward_train(self.logits, out=self.routed)
        d_logits = self.router.backward(self.logits, r, d_loss=torch.ones((), device=self.logits.device))
        self.w_router.addmm_(d_logits.t(), self.n32, alpha=-lr)
        return r.loss.clone(), r.counts.max().item() / self.T


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("hidden", 1024), ("inter", 512), ("experts", 32), ("topk", 4), ("tokens", 16), ("blocks", 3), ("train", 60)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    block = MoEBlock(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    h = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    y = 0.1 * torch.randn_like(h)
    for i in range(a.blocks):   # the same block over and over stands for a stack of them
        h, y = (t.clone() for t in block.step(h, y))
        print(f"block {i}: stream rms {h.float().square().mean().sqrt():.3f}, output rms {y.float().square().mean().sqrt():.3f}")
    big = MoEBlock(1024, a.hidden, a.inter, a.experts, a.topk, seed=1)
    big.w_router[0] += 0.02      # a router that prefers the first expert on a stream with a common component
    h = (torch.randn(1024, a.hidden, device="cuda") + 1.0).to(torch.bfloat16)
    y = torch.zeros_like(h)
    for i in range(a.train):
        loss, top = big.train_router(h, y, lr=1.0)
        if i % 10 == 0 or i == a.train - 1:
            print(f"router step {i}: loss {loss[0].item():.5f} (balance {loss[1].item():.5f}), largest expert takes {100 * top:.1f}% of tokens")
    assert block.experts.device_status() == moe.MOE_OK


if __name__ == "__main__":
    main()
