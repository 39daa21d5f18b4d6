"""A gated feed-forward layer, Y = (act(X Wg^T) * (X Wu^T)) Wd^T, trained and served with the library.

    python examples/feed_forward.py [--tokens 512] [--model 1024] [--hidden 2816]

Training: a few steps of gradient descent towards a fixed target on one batch, every product
and gradient by the library (bf16 weights and activations, float32 master weights held here).
Serving: the trained weights and each batch of activations in FP4 (E2M1, a scale per 32
elements), for a prompt and for single tokens.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_core_gemm_02_gb300 import binding as tc  # noqa: E402


class FeedForward:
    """Weights as the entry points take them: Wg, Wu (hidden x model), Wd (model x hidden)."""

    def __init__(self, model, hidden, act="silu", seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda n, k: torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5  # noqa: E731
        self.master = {"Wg": new(hidden, model), "Wu": new(hidden, model), "Wd": new(model, hidden)}
        self.act = act
        self.cast()

    def cast(self):
        self.Wg, self.Wu, self.Wd = (self.master[k].bfloat16() for k in ("Wg", "Wu", "Wd"))

    def forward(self, X):
        """Y, and what the backward pass needs."""
        M, N = X.shape[0], self.Wg.shape[0]
        G, U = (torch.empty((M, N), dtype=X.dtype, device=X.device) for _ in range(2))
        H = tc.gemm_gated(X, self.Wg, self.Wu, G=G, U=U, act=self.act, out=tc.OUT_BF16)
        return tc.gemm_bf16(H, self.Wd, out=tc.OUT_BF16), (X, G, U, H)

    def backward(self, dY, kept):
        """Gradients of X and of the three weights (float32)."""
        X, G, U, H = kept
        dH = tc.gemm_trans(dY, self.Wd, trans_b=True, out=tc.OUT_BF16)    # dY Wd
        dWd = tc.gemm_trans(dY, H, trans_a=True, trans_b=True)            # dY^T H
        # dG and dU take the place of G and U, which nothing reads after this
        dX, dWg, dWu, _, _ = tc.gemm_gated_backward(dH, G, U, X, self.Wg, self.Wu, dG=G, dU=U, act=self.act)
        return dX, {"Wg": dWg, "Wu": dWu, "Wd": dWd}

    def step(self, X, target, rate):
        """One step of gradient descent on half the squared distance of a token from its target (its
        mean over the tokens); returns that loss per element."""
        Y, kept = self.forward(X)
        diff = Y.float() - target
        loss = diff.square().mean() / 2
        _, grads = self.backward(diff.bfloat16(), kept)
        for k, g in grads.items():
            self.master[k] -= rate / X.shape[0] * g
        self.cast()
        return loss


class ServedFeedForward:
    """The layer with FP4 weights; activations are quantised on the way in and between the products."""

    def __init__(self, ffn):
        self.Wg, self.Wu, self.Wd = (tc.gemm_quantize_e2m1(w) for w in (ffn.Wg, ffn.Wu, ffn.Wd))
        self.act = ffn.act

    def __call__(self, X):
        H = tc.gemm_gated_e2m1(*tc.gemm_quantize_e2m1(X), *self.Wg, *self.Wu, act=self.act, out=tc.OUT_BF16)
        return tc.gemm_e2m1(*tc.gemm_quantize_e2m1(H), *self.Wd, out=tc.OUT_BF16)


def relative(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def run(tokens=512, model=1024, hidden=2816, steps=20, rate=0.05, say=print):
    """Losses over the steps and the served layer's distance from the trained one, per batch size."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((tokens, model), generator=gen, device="cuda").bfloat16()
    target = torch.randn((tokens, model), generator=gen, device="cuda") * 0.5
    ffn = FeedForward(model, hidden)
    losses = [ffn.step(X, target, rate) for _ in range(steps)]
    losses = [float(x) for x in losses]
    say(f"training, {tokens} tokens: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    served = ServedFeedForward(ffn)
    far = {}
    for m in sorted({tokens, 16, 1}):
        far[m] = relative(served(X[:m]), ffn.forward(X[:m])[0])
        say(f"serving in FP4, {m} tokens: {far[m]:.3f} from the bf16 layer (relative norm)")
    if tc.gemm_check_device_status() != tc.GEMM_OK:
        raise RuntimeError("a kernel reported an error")
    return losses, far


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--model", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    run(a.tokens, a.model, a.hidden, a.steps)
