"""The training example runs the new calls together and learns."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("act,bits", [("gelu", 32), ("gelu", 8), ("swiglu", 8)])
def test_example_learns(act, bits):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mixture_experts_topk_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_layer
    first, last = train_layer.train(steps=120, act=act, bits=bits, log=lambda s: None)
    # a layer that learns nothing stays at its first loss; noise between batches is a few per cent
    assert last < 0.7 * first, (first, last)


def test_layer_gradient_is_the_difference_quotient():
    """The whole layer's input gradient, gate included, against differences of
    the fp64 layer along a random direction, with the routing's choice fixed by
    a small step.  bf16 rounding of h, y, da and the results leaves the gradient
    within about 1e-2 of its norm; the quotient itself is exact to 1e-6."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import numpy as np
    from oracle import moe_oracle as O
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_layer
    layer = train_layer.Layer(96, 128, 6, 2, 96, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(96, 128, generator=gen, device="cuda").to(torch.bfloat16)
    dout = torch.randn(96, 128, generator=gen, device="cuda").to(torch.bfloat16)
    layer.forward(x)
    dx = layer.backward(x, dout).double().cpu().numpy()
    f = {k: v.double().cpu().numpy() for k, v in layer.copy.items()}
    x64, d64, ids = x.double().cpu().numpy(), dout.double().cpu().numpy(), layer.ids.cpu().numpy()

    def loss(xx):
        l = O.gate_logits(xx, f["Wg"])
        s = np.take_along_axis(l, ids, 1)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        d = O.dispatch(ids, 6, 0)
        y = O.expert_outputs(xx, d, f["W1"], f["W2"], ids=ids)
        return float((d64 * O.combine(y, d["pos"], w)).sum())

    rng = np.random.default_rng(6)
    for _ in range(4):
        way = rng.standard_normal(x64.shape)
        way /= np.linalg.norm(way)
        got = (loss(x64 + 1e-4 * way) - loss(x64 - 1e-4 * way)) / 2e-4
        assert abs(got - float((dx * way).sum())) <= 1e-2 * np.linalg.norm(dx), got
