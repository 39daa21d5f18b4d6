"""The feed-forward example end to end (needs a GB300): its gradients against 64-bit autograd,
training that lowers the loss, and the served FP4 layer."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_lowers_the_loss_and_fp4_serves(example):
    losses, far = example.run(tokens=200, model=256, hidden=672, steps=12, say=lambda *_: None)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    # E2M1 rounds an element by at most a sixth of it within a binade (1/12 on average), two
    # operands and two layers deep: well under half of the result
    assert set(far) == {200, 16, 1} and all(v < 0.5 for v in far.values())


def test_layer_gradients_against_autograd(example):
    """The whole layer: each 16-bit tensor on the way (G, U, H, dH, dG, dU) is rounded once to
    bf16, at most 2^-9 of each element; six such roundings and the slope's own change with G
    keep every gradient within 2^-5 of its norm."""
    ffn = example.FeedForward(256, 360)
    gen = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn((96, 256), generator=gen, device="cuda").bfloat16()
    dY = torch.randn((96, 256), generator=gen, device="cuda").bfloat16()
    _, kept = ffn.forward(X)
    dX, grads = ffn.backward(dY, kept)
    x, wg, wu, wd = (t.double().requires_grad_() for t in (X, ffn.Wg, ffn.Wu, ffn.Wd))
    y = (torch.nn.functional.silu(x @ wg.T) * (x @ wu.T)) @ wd.T
    want = torch.autograd.grad(y, (x, wg, wu, wd), dY.double())
    for got, ref in zip((dX, grads["Wg"], grads["Wu"], grads["Wd"]), want):
        assert (got.double() - ref).norm() <= 2.0 ** -5 * ref.norm()
