"""The expert block of examples/expert_block_16bit.py: its gradients against
automatic differentiation of the same block in 64 bits, its steps, and a step
captured in a CUDA graph.

Bounds.  The block rounds to bf16 (2^-8 relative) at n, act, y, dy, d_act, d_up
and dn, and its weights are given in bf16: a gradient passes at most six such
roundings on its way, each independent, so its error in the 2-norm stays within
6 * 2^-8 of its size.
"""
import importlib.util
import os

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
REL = 6 * 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_block_16bit.py")
    spec = importlib.util.spec_from_file_location("expert_block_16bit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def exact(example, block, x, sizes, gate, dx_out):
    w = {k: v.double().requires_grad_() for k, v in block.weights.items()}
    x, gate = x.double().requires_grad_(), gate.double().requires_grad_()
    unit = lambda z: z * (z.pow(2).mean(1, keepdim=True) + example.EPS).rsqrt()  # noqa: E731
    n = unit(x) * w["w_pre"]
    y = torch.cat([torch.nn.functional.silu(a @ w["w1"][g].t()) @ w["w2"][g].t()
                   for g, a in enumerate(n.split(sizes.tolist()))])
    out = x + block.scale * gate[:, None] * unit(y) * w["w_post"]
    out.backward(dx_out.double())
    return out.detach(), {**{k: v.grad for k, v in w.items()}, "x": x.grad, "gate": gate.grad}


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("rows,hidden,ffn,experts", [(300, 256, 328, 4), (65, 136, 72, 8), (3, 64, 64, 4)])
def test_gradients(example, rows, hidden, ffn, experts):
    block = example.Block(rows, hidden, ffn, experts, scale=0.5)
    x, sizes, gate, dx_out = example.batch(rows, hidden, experts)
    out = block.forward(x, sizes, gate)
    dx, dgate = block.backward(x, gate, dx_out)
    want, grads = exact(example, block, x, sizes, gate, dx_out)
    assert off(out, want) <= REL
    for k, v in block.grads.items():
        assert off(v, grads[k]) <= REL, k
    assert off(dx, grads["x"]) <= REL and off(dgate, grads["gate"]) <= REL


def test_steps_and_graph(example):
    block = example.Block(200, 128, 200, 4, max_norm=0.01)
    data = example.batch(200, 128, 4)
    losses = [float(block.step(*data, lr=50.0)) for _ in range(5)]
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert float(block.norm) > 0.01  # clipped: the gradients' norm is the limit
    total = sum(float(g.double().pow(2).sum()) for g in block.grads.values()) ** 0.5
    assert abs(total - 0.01) < 1e-5
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = block.step(*data, lr=50.0)
    graph.replay()
    first = float(loss)
    for _ in range(3):
        graph.replay()
    assert float(loss) < first < losses[-1]
