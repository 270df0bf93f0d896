"""A mixture-of-experts layer on 16-bit tensors, trained with libmxg's operators.

    l  = x Wr^T                                   the router's logits, fp32
    e, w = the k best experts of a token and their weights; rows sorted by expert
    g, u = x[row] W1[e]^T                         grouped product, gate and up side by side
    y  = sum_j w_j (silu(g) u) W2[e_j]^T
    loss = mean((y - target)^2) + balance loss

The activation's inputs are kept in 8 bits; the backward pass makes silu(g) u again from them.
``Layer.step`` runs all of it forward and backward, and clips the gradients of all weights as one
vector.  Everything but the loss and the update is a call of the library.

    python examples/moe_layer_16bit.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_block_gb300 import mxg  # noqa: E402

BF = torch.bfloat16


class Layer:
    """A layer's weights (bf16), their gradients, and the buffers of a step of `tokens` tokens."""

    def __init__(self, tokens, hidden, ffn, experts, k, balance=0.01, max_norm=1.0, device="cuda", seed=0):
        self.T, self.D, self.F, self.E, self.k = tokens, hidden, ffn, experts, k
        self.balance, self.max_norm = balance, max_norm
        self.R = tokens * k  # rows that the experts get at most
        gen = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731

        def weight(*shape):
            w = torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5
            return w.to(BF)
        self.weights = {"wr": weight(experts, hidden), "w1": weight(experts, 2 * ffn, hidden),
                        "w2": weight(experts, hidden, ffn)}
        self.grads = {k: torch.zeros_like(v, dtype=torch.float32) for k, v in self.weights.items()}
        self.grad_list = mxg.grad_list(self.grads.values())
        self.grad_ws, self.norm = mxg.alloc_grad_workspace(device), new(1, dtype=torch.float32)
        # one group of all tokens, for the router's products
        self.all = torch.tensor([tokens, 0, tokens], dtype=torch.int64, device=device)
        self.one = torch.ones(1, device=device)
        # routing
        i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
        f32 = lambda *s: new(*s, dtype=torch.float32)  # noqa: E731
        self.logits, self.dlogits = f32(tokens, experts), f32(tokens, experts)
        self.expert, self.row_of, self.counts = i32(tokens, k), i32(tokens, k), i32(experts)
        self.weight, self.dweight = f32(tokens, k), f32(tokens, k)
        self.loss, self.slope = f32(1), f32(experts)
        self.groups = mxg.alloc_offsets(experts, device)
        self.route_ws = mxg.alloc_route_workspace(tokens, experts, k, device)
        # rows
        self.xs, self.rows, self.drows, self.dxs = (new(self.R, hidden) for _ in range(4))
        self.gu, self.dgu = new(self.R, 2 * ffn), new(self.R, 2 * ffn)
        self.h, self.dh = new(self.R, ffn), new(self.R, ffn)
        self.q, self.sf = mxg.alloc_act_checkpoint(self.R, ffn, True, device)
        self.y, self.dx = new(tokens, hidden), new(tokens, hidden)

    def _product(self, mode, a, b, out, n, k):
        mxg.mxg_grouped_gemm_16bit(mode, a, b, self.groups, self.E, self.R, n, k, C=out)

    def forward(self, x, mask=None):
        """x [tokens, hidden], mask [tokens] (0: padding) or None -> y."""
        w, F = self.weights, self.F
        mxg.mxg_grouped_gemm_16bit(mxg.MXG_FPROP_TN, x, w["wr"], self.all, 1, self.T, self.E, self.D,
                                   C=self.logits)
        mxg.mxg_route(self.logits, self.expert, self.weight, self.counts, mask=mask, balance=self.balance,
                      loss=self.loss, slope=self.slope, row_of=self.row_of, group_ws=self.groups,
                      last_dim=self.D, workspace=self.route_ws)
        mxg.mxg_dispatch(x, self.row_of, self.xs)
        self._product(mxg.MXG_FPROP_TN, self.xs, w["w1"], self.gu, 2 * F, self.D)
        mxg.mxg_gated_act(self.gu[:, :F], self.h, up=self.gu[:, F:], q=self.q, sf=self.sf,
                          group_ws=self.groups, G=self.E)
        self._product(mxg.MXG_FPROP_TN, self.h, w["w2"], self.rows, self.D, F)
        mxg.mxg_combine(self.rows, self.row_of, self.y, weight=self.weight)
        return self.y

    def backward(self, x, dy):
        """The gradient of x for dy, that of y, and 1, that of the balance loss; the weights' in
        self.grads."""
        w, g, F = self.weights, self.grads, self.F
        mxg.mxg_combine_backward(dy, self.row_of, self.weight, self.drows, y_rows=self.rows,
                                 dweight=self.dweight)
        self._product(mxg.MXG_DGRAD_NN, self.drows, w["w2"], self.dh, self.D, F)
        mxg.mxg_gated_act_backward(self.q, self.sf, self.dh, self.dgu[:, :F], dup=self.dgu[:, F:],
                                   h=self.h, group_ws=self.groups, G=self.E)
        self._product(mxg.MXG_WGRAD_NT, self.drows, self.h, g["w2"], self.D, F)
        self._product(mxg.MXG_WGRAD_NT, self.dgu, self.xs, g["w1"], 2 * F, self.D)
        self._product(mxg.MXG_DGRAD_NN, self.dgu, w["w1"], self.dxs, 2 * F, self.D)
        mxg.mxg_combine(self.dxs, self.row_of, self.dx)  # what dispatch's gradient is
        # the router: what its logits get from the weights and from the balance loss
        mxg.mxg_route_backward(self.logits, self.expert, self.dlogits, dweight=self.dweight,
                               slope=self.slope, dloss=self.one)
        dl = self.dlogits.to(BF)
        mxg.mxg_grouped_gemm_16bit(mxg.MXG_WGRAD_NT, dl, x, self.all, 1, self.T, self.E, self.D, C=g["wr"])
        mxg.mxg_grouped_gemm_16bit(mxg.MXG_DGRAD_NN, dl, w["wr"], self.all, 1, self.T, self.E, self.D,
                                   beta=self.one, C=self.dx)
        return self.dx

    def step(self, x, target, lr, mask=None):
        """One step of gradient descent; returns the loss."""
        error = self.forward(x, mask).float() - target.float()
        self.backward(x, (error * (2 / error.numel())).to(BF))
        mxg.mxg_grad_clip(self.grad_list, self.max_norm, self.norm, self.grad_ws)
        for k, v in self.weights.items():
            v.copy_(v.float() - lr * self.grads[k])
        return error.square().mean() + self.loss[0]


def batch(tokens, hidden, device="cuda", seed=1):
    """Tokens, a target to fit, and a mask: the last tenth is padding."""
    gen = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=gen, device=device).to(BF)
    target = torch.randn(tokens, hidden, generator=gen, device=device).to(BF)
    mask = (torch.arange(tokens, device=device) < tokens - tokens // 10).to(torch.uint8)
    return x, target, mask


def main():
    tokens, hidden, ffn, experts, k = 1000, 512, 704, 16, 4
    layer = Layer(tokens, hidden, ffn, experts, k)
    x, target, mask = batch(tokens, hidden)
    for i in range(10):
        loss = layer.step(x, target, 20.0, mask)
        print("step %d: loss %.4f, balance %.4f, gradient norm %.4f"
              % (i, float(loss), float(layer.loss), float(layer.norm)))


if __name__ == "__main__":
    main()
