"""The training-step example: its gradients against autograd in float64, and that it learns."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("moe_training_step", os.path.join(ROOT, "examples",
                                                                                   "moe_training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_layer_gradients_match_autograd(example):
    import torch
    p, T, H, E, K = 3, 20, 16, 6, 2
    layer = example.MoeLayer(p, H, E, K, seed=4)
    x = torch.randn((p, T, H), device="cuda")
    dy = torch.randn((p, T, H), device="cuda")
    y = layer.forward(x)
    got = layer.backward(dy)
    x64, r64, w64 = (t.double().cpu().requires_grad_() for t in (x, layer.router, layer.experts))
    ids = layer.ids.long().cpu()
    weights = torch.softmax(torch.gather(x64 @ r64, 2, ids), dim=-1)
    want_y = sum(weights[..., k, None] * (x64[:, :, None] @ w64[ids[..., k]])[:, :, 0] for k in range(K))
    want_y.backward(dy.double().cpu())
    # every value is a sum of at most H * T * p products in float32 (of factors that are such sums themselves)
    n = 4 * H * T * p
    for a, b in zip((y, *got), (want_y.detach(), x64.grad, r64.grad, w64.grad)):
        assert float((a.double().cpu() - b).abs().max()) <= n * 2.0 ** -24 * float(b.abs().max())


@pytest.mark.parametrize("bits", [32, 8])
def test_training_reduces_the_loss(example, bits):
    losses = example.train(60, bits, say=None)
    assert losses[-1] < 0.5 * losses[0] and all(x == x for x in losses)
