"""What the bounds of gemm_orthogonalize's tests accept and refuse, on the CPU: the steps emulated in 64 bits
with the roundings of the kernels, and with mistakes planted in them."""
import pytest
import torch

from test_gpu_orthogonalize import EPS, MUON, QUINTIC, SINGULAR, recurrence, spread_matrix

SCALE = 4096.0  # of the float16 iterates and products


def one(x):
    return (x * SCALE).half().double() / SCALE


def two(x):
    return one(x) + one(x - one(x))


def emulate(x, coefs, steps, iterate, product):
    """The steps with the iterates and the products rounded by these functions, float32 at the end."""
    a, b, c = coefs
    x = x.double()
    x = iterate(x / (x.norm() + EPS))
    for i in range(steps):
        p = product(x @ x.T)
        x = a * x + product(b * p + c * (p @ p)) @ x
        x = iterate(x) if i < steps - 1 else x.float().double()
    return x


@pytest.mark.parametrize("coefs", [QUINTIC, MUON])
@pytest.mark.parametrize("steps", [1, 2])
def test_few_steps(coefs, steps):
    """The elementwise bound of float32 results takes operands in two parts and refuses iterates in one."""
    x = spread_matrix()
    want, bound = recurrence(x, coefs, steps, EPS, torch.float32)
    assert (emulate(x, coefs, steps, two, two) - want).norm() < bound / 10
    assert (emulate(x, coefs, steps, one, two) - want).norm() > 2 * bound


def test_singular_values():
    """After 14 steps: products in one part are refused."""
    x = spread_matrix()
    want = torch.linalg.svdvals(recurrence(x, QUINTIC, 14, EPS, torch.float32)[0])
    off = lambda *r: (torch.linalg.svdvals(emulate(x, QUINTIC, 14, *r)) - want).abs().max()  # noqa: E731
    assert off(two, two) < SINGULAR / 10
    assert off(two, one) > 10 * SINGULAR and off(one, one) > 10 * SINGULAR
