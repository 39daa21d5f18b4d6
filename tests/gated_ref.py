"""Plain 64-bit forms of the gated operators, and the bounds the GPU results are held to.

Sums: the tensor cores add K in steps of 16 into a float32 accumulator; each step
is taken to lose at most two units (2^-22) of a running sum that never exceeds
T = sum_k |a||b|, so |sum - exact| <= sum_bound(K) * T.

Activation: float32 with the fast exponential (documented error: 2 + 1.173 |x|
units of 2^-23 for e^x) and division (2 units), whose argument y itself carries
a couple of roundings: relative error at most (16 + 8 |y|) 2^-23; forms with
1 + erf or 1 + tanh cancel for negative g, an absolute error of at most
4 * 2^-23 |g|.  A 16-bit output adds half a unit in its last place (bf16 2^-8 |x|
with its next power of two, f16 2^-11 |x| and 2^-25 below its normal range).
"""
import math

import numpy as np
import torch

from tensor_core_gemm_02_gb300.workloads import OUT_BF16, OUT_F16, OUT_F32, OUT_TORCH

ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
# largest slope of each activation (silu 1.0999, gelu 1.1290, gelu_tanh 1.1291, sigmoid 1/4)
SLOPE = {"silu": 1.11, "gelu": 1.14, "gelu_tanh": 1.14, "relu": 1.0, "sigmoid": 0.25}
C0 = math.sqrt(2.0 / math.pi)


def act64(name, g):
    if name == "silu":
        return g * torch.special.expit(g)
    if name == "gelu":
        return 0.5 * g * torch.special.erfc(-g / math.sqrt(2.0))
    if name == "gelu_tanh":
        return g * torch.special.expit(2 * C0 * (g + 0.044715 * g ** 3))
    if name == "relu":
        return torch.clamp(g, min=0.0)
    return torch.special.expit(g)


def slope64(name, g):
    if name == "silu":
        p = torch.special.expit(g)
        return p * (1 + g * (1 - p))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        p = torch.special.expit(2 * C0 * (g + 0.044715 * g ** 3))
        return p + g * p * (1 - p) * 2 * C0 * (1 + 3 * 0.044715 * g * g)
    if name == "relu":
        return (g > 0).double()
    p = torch.special.expit(g)
    return p * (1 - p)


def argument(name, g, slope=False):
    """|y| of the exponential inside the activation (or its slope; gelu itself has only erf)."""
    if name == "relu":
        return torch.zeros_like(g)
    if name == "gelu":
        return 0.5 * g * g if slope else torch.zeros_like(g)
    if name == "gelu_tanh":
        return (2 * C0 * (g + 0.044715 * g ** 3)).abs()
    return g.abs()


def sum_bound(K):
    return (K / 16 + 2) * 2.0 ** -22


def rounding(ref, out):
    if out == OUT_F32:
        return ref.abs() * 2.0 ** -24 + 2.0 ** -149
    if out == OUT_BF16:
        return ref.abs() * 2.0 ** -8
    return ref.abs() * 2.0 ** -11 + 2.0 ** -25


def gated64(A, Bg, Bu, act):
    """(D, G, U, T of G, T of U) in 64 bits, on the CPU."""
    a, bg, bu = A.cpu().double(), Bg.cpu().double(), Bu.cpu().double()
    g, u = a @ bg.T, a @ bu.T
    return act64(act, g) * u, g, u, a.abs() @ bg.abs().T, a.abs() @ bu.abs().T


def gated_bound(act, K, d, g, u, tg, tu, out):
    eg, eu = sum_bound(K) * tg, sum_bound(K) * tu
    a, lip = act64(act, g).abs(), SLOPE[act]
    y = argument(act, g.abs() + eg)
    err = lip * eg * (u.abs() + eu) + a * eu
    err = err + a * u.abs() * (16 + 8 * y) * 2.0 ** -23 + 4 * 2.0 ** -23 * g.abs() * (u.abs() + eu)
    return err + rounding(d.abs() + err, out)


def assert_close(got, ref, bound, what=""):
    got = got.detach().cpu().double()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = torch.nonzero(bad)[:4].tolist()
        worst = (err / bound.clamp(min=1e-300)).max().item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first {i}, worst "
                             f"{worst:.3g} of it")


def wide(rows, cols, dtype, gen, scale=1.0, pad=8, device="cuda", exact=False):
    """A rows x cols slice of a wider buffer whose padding is NaN, rows a multiple of 8 elements
    apart; exact: quarter-integers in [-1, 1]."""
    ld = (cols + 7) // 8 * 8 + pad
    buf = torch.full((max(rows, 1), ld), float("nan"), dtype=torch.float32)
    x = (torch.randint(-4, 5, (rows, cols), generator=gen).float() / 4 if exact
         else torch.randn((rows, cols), generator=gen)) * scale
    buf[:rows, :cols] = x
    return buf.to(dtype).to(device)[:rows, :cols]


def out_dtype(out):
    return OUT_TORCH[out]


# ---------------------------------------------------------------- E2M1

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize64(x):
    """(codes M x K, scales M x K/32, values M x K) of a float64 array, element by element from the
    definition: the nearest level, the even code of two equally near."""
    x = np.asarray(x, np.float64)
    m, k = x.shape
    b = x.reshape(m, k // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=2))
    _, e = np.frexp(top)  # top = f 2^e with f in [1/2, 1)
    s = np.where(top > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0).astype(np.int64)
    z = np.where(bad[:, :, None], 0.0, np.ldexp(np.where(np.isfinite(b), b, 0.0), (127 - s)[:, :, None]))
    dist = np.abs(np.minimum(np.abs(z), 6.0)[..., None] - LEVELS)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), np.argmax(even, -1), np.argmax(near, -1))
    minus = np.signbit(z)
    v = np.ldexp(np.where(minus, -LEVELS[code], LEVELS[code]), (s - 127)[:, :, None])
    v = np.where(bad[:, :, None], np.nan, v)
    code = np.where(minus, code + 8, code)
    return code.reshape(m, k), np.where(bad, 255, s), v.reshape(m, k)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
