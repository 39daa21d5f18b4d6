"""A layer of gated experts, trained with the library and its weights' updates orthogonalised.

    python examples/experts.py [--tokens 1024] [--model 1024] [--hidden 704] [--experts 16] [--choices 2]

Each token goes to the experts its router's scores are highest for, weighted by their softmax:
    Y[t] = sum over its experts e of w[t][e] (silu(X[t] Wg_e^T) * (X[t] Wu_e^T)) Wd_e^T.
The assignments are grouped by expert (gemm_group_rows), the tokens' rows gathered by the products
themselves (gemm_grouped); the backward pass takes the same groups (gemm_grouped with trans_b,
gemm_grouped_weights).  A step moves every expert's three matrices by their momentum's
orthogonalised form (gemm_orthogonalize on the whole stack).  The scores are given; router and
elementwise parts are torch's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_core_gemm_02_gb300 import binding as tc  # noqa: E402


class Experts:
    """Weights as the entry points take them: Wg, Wu (experts x hidden x model), Wd (experts x model x hidden)."""

    def __init__(self, experts, model, hidden, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda n, k: torch.randn((experts, n, k), generator=gen, device="cuda") * k ** -0.5  # noqa: E731
        self.master = {"Wg": new(hidden, model), "Wu": new(hidden, model), "Wd": new(model, hidden)}
        self.momentum = {k: torch.zeros_like(w) for k, w in self.master.items()}
        self.experts, self.dtype = experts, dtype
        self.out = tc.OUT_BF16 if dtype == torch.bfloat16 else tc.OUT_F16
        self.cast()

    def cast(self):
        self.Wg, self.Wu, self.Wd = (self.master[k].to(self.dtype) for k in ("Wg", "Wu", "Wd"))

    def forward(self, X, ids, w):
        """Y (float32) for tokens X, their experts ids and weights w (tokens x choices); and what
        the backward pass needs."""
        off, order, rows = tc.gemm_group_rows(ids, self.experts)
        G = tc.gemm_grouped(X, self.Wg, off, idx=rows, out=self.out)
        U = tc.gemm_grouped(X, self.Wu, off, idx=rows, out=self.out)
        H = (torch.nn.functional.silu(G.float()) * U.float()).to(self.dtype)
        O = tc.gemm_grouped(H, self.Wd, off)
        # where assignment (t, j) lies among the groups
        place = torch.empty_like(order).scatter_(0, order.long(), torch.arange(len(order), dtype=order.dtype, device=X.device))
        place = place.long().view(ids.shape)
        Y = (O[place] * w[:, :, None]).sum(dim=1)
        return Y, (X, w, off, order.long(), rows.long(), place, G, U, H, O)

    def backward(self, dY, kept):
        """Gradients of X, of the weights w and of the three stacks (float32)."""
        X, w, off, order, rows, place, G, U, H, O = kept
        dw = (O[place] * dY[:, None, :]).sum(dim=2)
        dO = (dY[rows] * w.flatten()[order][:, None]).to(self.dtype)
        dH = tc.gemm_grouped(dO, self.Wd, off, trans_b=True)
        s = torch.sigmoid(G.float())
        dG = (dH * U.float() * s * (1 + G.float() * (1 - s))).to(self.dtype)
        dU = (dH * G.float() * s).to(self.dtype)
        dXs = tc.gemm_grouped(dG, self.Wg, off, trans_b=True) + tc.gemm_grouped(dU, self.Wu, off, trans_b=True)
        Xs = X[rows]
        return dXs[place].sum(dim=1), dw, {"Wg": tc.gemm_grouped_weights(dG, Xs, off),
                                           "Wu": tc.gemm_grouped_weights(dU, Xs, off),
                                           "Wd": tc.gemm_grouped_weights(dO, H, off)}

    def step(self, X, ids, w, target, rate, decay=0.9):
        """One step towards the target; returns half the mean squared distance."""
        Y, kept = self.forward(X, ids, w)
        diff = Y - target
        _, _, grads = self.backward(diff / X.shape[0], kept)
        for k, g in grads.items():
            self.momentum[k].mul_(decay).add_(g)
            n, m = g.shape[1:]
            self.master[k] -= rate * (n / m) ** 0.5 * tc.gemm_orthogonalize(self.momentum[k].to(self.dtype)).float()
        self.cast()
        return diff.square().mean() / 2


def route(scores, choices):
    """The experts of each token and their weights."""
    w, ids = scores.topk(choices, dim=1)
    return ids.to(torch.int32), torch.softmax(w, dim=1)


def run(tokens=1024, model=1024, hidden=704, experts=16, choices=2, steps=10, rate=0.02, say=print):
    """The losses over the steps."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((tokens, model), generator=gen, device="cuda").bfloat16()
    target = torch.randn((tokens, model), generator=gen, device="cuda") * 0.5
    ids, w = route(torch.randn((tokens, experts), generator=gen, device="cuda"), choices)
    layer = Experts(experts, model, hidden)
    losses = [float(layer.step(X, ids, w, target, rate)) for _ in range(steps)]
    say(f"training, {tokens} tokens, {choices} of {experts} experts each: loss {losses[0]:.4f} -> {losses[-1]:.4f} "
        f"in {steps} steps")
    if tc.gemm_check_device_status() != tc.GEMM_OK:
        raise RuntimeError("a kernel reported an error")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 1024), ("model", 1024), ("hidden", 704), ("experts", 16), ("choices", 2),
                          ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    run(**vars(ap.parse_args()))
