"""Training an expert block on 16-bit tensors with libmxg's operators.

The block, on tokens that the router has sorted by expert (one expert a token,
its probability the row's gate):

    n  = norm(x) . w_pre
    y  = silu(n W1[g]^T) W2[g]^T                    grouped products
    x' = x + scale * gate * norm(y) . w_post

``Block.step`` runs it forward and backward on a batch and clips the gradients
of all weights as one vector.  Everything but the activation and the update is a
call of the library.

    python examples/expert_block_16bit.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_block_gb300 import mxg  # noqa: E402

EPS = 1e-6


def silu_and_slope(u: torch.Tensor):
    """silu(u) and its derivative, in fp32."""
    s = torch.sigmoid(u)
    return u * s, s * (1 + u * (1 - s))


class Block:
    """An expert block's weights (bf16), their gradients, and the buffers of a step of at most
    `rows` tokens."""

    def __init__(self, rows, hidden, ffn, experts, scale=1.0, max_norm=1.0, device="cuda", seed=0):
        self.R, self.D, self.F, self.G = rows, hidden, ffn, experts
        self.scale, self.max_norm = scale, max_norm
        gen = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731

        def weight(*shape):
            w = torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5
            return w.to(torch.bfloat16)
        self.weights = {"w1": weight(experts, ffn, hidden), "w2": weight(experts, hidden, ffn),
                        "w_pre": torch.ones(hidden, dtype=torch.bfloat16, device=device),
                        "w_post": torch.ones(hidden, dtype=torch.bfloat16, device=device)}
        # gradients are accumulated in fp32
        self.grads = {k: torch.zeros_like(v, dtype=torch.float32) for k, v in self.weights.items()}
        self.grad_list = mxg.grad_list(self.grads.values())
        self.grad_ws = mxg.alloc_grad_workspace(device)
        self.norm = new(1, dtype=torch.float32)
        self.norm_ws = mxg.alloc_block_norm_workspace(rows, hidden, device)
        self.groups = mxg.alloc_offsets(experts, device)
        self.n, self.y, self.x_out = new(rows, hidden), new(rows, hidden), new(rows, hidden)
        self.up = new(rows, ffn, dtype=torch.float32)
        self.dx, self.dy, self.dn = new(rows, hidden), new(rows, hidden), new(rows, hidden)
        self.d_act = new(rows, ffn)
        self.dgate = new(rows, dtype=torch.float32)

    def _product(self, mode, a, b, out, n, k):
        mxg.mxg_grouped_gemm_16bit(mode, a, b, self.groups, self.G, self.R, n, k, C=out)

    def forward(self, x, sizes, gate):
        """x [rows, hidden] sorted by expert, sizes [experts], gate fp32 [rows] -> x'."""
        w = self.weights
        mxg.mxg_group_offsets_unaligned(sizes, 1, self.D, self.R, self.groups)
        mxg.mxg_block_norm(x, w_pre=w["w_pre"], n_out=self.n, eps=EPS)
        self._product(mxg.MXG_FPROP_TN, self.n, w["w1"], self.up, self.F, self.D)
        act, self.slope = silu_and_slope(self.up)
        self.act = act.to(torch.bfloat16)
        self._product(mxg.MXG_FPROP_TN, self.act, w["w2"], self.y, self.D, self.F)
        mxg.mxg_block_norm(x, self.y, w_post=w["w_post"], gate=gate, gate_mode=mxg.MXG_GATE_ROW,
                           res_scale=self.scale, x_out=self.x_out, eps=EPS)
        return self.x_out

    def backward(self, x, gate, dx_out):
        """The gradients of x and of the gate for dx_out, that of x'; the weights' in self.grads."""
        w, g = self.weights, self.grads
        mxg.mxg_block_norm_backward(self.x_out, self.y, w_post=w["w_post"], gate=gate,
                                    gate_mode=mxg.MXG_GATE_ROW, res_scale=self.scale, eps=EPS,
                                    dx_out=dx_out, dx=self.dx, dy=self.dy, dw_post=g["w_post"],
                                    dgate=self.dgate, workspace=self.norm_ws)
        self._product(mxg.MXG_WGRAD_NT, self.dy, self.act, g["w2"], self.D, self.F)
        self._product(mxg.MXG_DGRAD_NN, self.dy, w["w2"], self.d_act, self.D, self.F)
        d_up = (self.d_act.float() * self.slope).to(torch.bfloat16)
        self._product(mxg.MXG_WGRAD_NT, d_up, self.n, g["w1"], self.F, self.D)
        self._product(mxg.MXG_DGRAD_NN, d_up, w["w1"], self.dn, self.F, self.D)
        # the norm before the block; dx already holds what came past the block
        mxg.mxg_block_norm_backward(x, w_pre=w["w_pre"], eps=EPS, dx_out=self.dx, dn=self.dn,
                                    dx=self.dx, dw_pre=g["w_pre"], workspace=self.norm_ws)
        return self.dx, self.dgate

    def step(self, x, sizes, gate, target, lr):
        """One step of gradient descent on mean((x' - target)^2); returns the loss."""
        error = self.forward(x, sizes, gate).float() - target.float()
        self.backward(x, gate, (error * (2 / error.numel())).to(torch.bfloat16))
        mxg.mxg_grad_clip(self.grad_list, self.max_norm, self.norm, self.grad_ws)
        for k, v in self.weights.items():
            v.copy_(v.float() - lr * self.grads[k])
        return error.square().mean()


def batch(rows, hidden, experts, device="cuda", seed=1):
    """Tokens sorted by expert, with group sizes of any value, and a target to fit."""
    gen = torch.Generator(device=device).manual_seed(seed)
    logits = torch.randn(rows, experts, generator=gen, device=device)
    p, expert = logits.softmax(1).max(1)
    order = torch.argsort(expert, stable=True)
    x = torch.randn(rows, hidden, generator=gen, device=device).to(torch.bfloat16)
    target = torch.randn(rows, hidden, generator=gen, device=device).to(torch.bfloat16)
    sizes = torch.bincount(expert, minlength=experts).to(torch.int32)
    return x[order].contiguous(), sizes, p[order].contiguous(), target[order].contiguous()


def main():
    rows, hidden, ffn, experts = 1000, 512, 1408, 8
    block = Block(rows, hidden, ffn, experts)
    x, sizes, gate, target = batch(rows, hidden, experts)
    for i in range(10):
        loss = block.step(x, sizes, gate, target, lr=20.0)
        print("step %d: loss %.4f, gradient norm %.4f" % (i, float(loss), float(block.norm)))


if __name__ == "__main__":
    main()
