"""The gated form's activations themselves, on the GPU (needs a GB300).

G and U are exact in float32 here (few dyadic terms; relu and gemm_f16 show that first) and
D is float32, so what is left is the activation's own error.  Bounds, in units u = 2^-23 of
the value, from the instructions' documented errors (the base-2 exponential 2 u, the
reciprocal 1 u; a rounding 1/2 u, a constant 1/4 u):

  sigmoid     the argument log2(e) x is off by 3/4 u of itself, the sum and the reciprocal add 3/2,
              and the product by U 1/2: (4 + 3/4 |x|) u, taken as (5 + |x|) u
  silu        one product more: the same bound
  gelu_tanh   the argument y, a sum of terms of one sign, is off by at most 2 u of itself:
              (5 + 3 |y|) u
  gelu        exp(-g^2 / 2), two roundings and a constant in its argument: (2 + 5/4 y) u with
              y = g^2 / 2; the polynomial in t 4 u as evaluated in float32 with t rounded
              correctly, 2 more for t's reciprocal, and four products: (12 + 2 y) u

Exponentials' reciprocals below 2^-126 are flushed: with |g| <= 12 and |U| = 1 less than
2^-120 of D.  (gelu's exponential reaches that at g = -13.)
"""
import math

import pytest
import torch

import gated_ref as ref
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding
from tensor_core_gemm_02_gb300.workloads import OUT_F16, OUT_F32

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
F16 = torch.float16
FORMS = {"skinny": (2, 0), "single64": (1, 64), "single256": (1, 256), "pair": (3, 256)}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK


def bound(act, g):
    """Relative error allowed at g."""
    if act == "relu":
        return torch.full_like(g, U)
    if act == "gelu":
        return (12 + g * g) * U
    if act == "gelu_tanh":
        return (5 + 3 * (2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)).abs()) * U
    return (5 + g.abs()) * U


def check(got, act, g, u, what):
    want = ref.act64(act, g) * u
    err = (got.cpu().double() - want).abs()
    allowed = bound(act, g) * want.abs() + 2.0 ** -120
    bad = ~(err <= allowed)
    if bad.any():
        worst = int((err / allowed).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at g = {g.flatten()[worst]:.6f}: "
                             f"{(err / allowed).max():.3g} of the bound, relative error "
                             f"{(err / want.abs()).flatten()[worst]:.3g}")


def sweep(n):
    """A (rows +-[1, 2^-11]), Bg and Bu with G = +-g exactly, g swept over [-12, 12] in multiples of
    2^-19 (a float16 and 2^-11 of another), and U = 1; and G."""
    g = torch.round(torch.linspace(-12, 12, n, dtype=torch.float64) * 2 ** 19) / 2 ** 19
    high = g.half()
    low = ((g - high.double()) * 2 ** 11).half()
    assert torch.equal(high.double() + low.double() / 2 ** 11, g)
    B = torch.zeros((2, n, 8), dtype=F16)
    B[0, :, 0], B[0, :, 1], B[1, :, 0] = high, low, 1
    A = torch.zeros((16, 8), dtype=F16)
    A[:, 0], A[:, 1] = 1, 2.0 ** -11
    A[1::2] *= -1
    sign = torch.where(torch.arange(16) % 2 == 0, 1.0, -1.0).double()[:, None]
    return A.cuda(), B[0].cuda(), B[1].cuda(), sign * g, sign.expand(16, n)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", ref.ACTS)
def test_relative_error_over_a_sweep(act, form):
    A, Bg, Bu, g, u = sweep(20001)
    assert torch.equal(binding.gemm_f16(A, Bg).cpu().double(), g)  # G is exact
    binding.gemm_debug_force_tile(*FORMS[form])
    assert torch.equal(binding.gemm_gated(A, Bg, Bu, act="relu").cpu().double(), g.clamp(min=0) * u)
    check(binding.gemm_gated(A, Bg, Bu, act=act, out=OUT_F32), act, g, u, form)


@pytest.mark.parametrize("act", ["gelu"])
@pytest.mark.parametrize("M,bn", [(16, 0), (130, 128), (130, 256)])
def test_relative_error_fp4(act, M, bn):
    """Both operands FP4: sums of a few dyadic terms, most of them within |g| <= 12."""
    N, K = 3000, 288  # (more than 256 elements: few rows take the swap-AB kernel)
    r = torch.Generator().manual_seed(M)
    levels = torch.tensor([*ref.LEVELS, *-ref.LEVELS], dtype=torch.float64)

    def make(rows, scale):
        codes = torch.zeros((rows, K), dtype=torch.uint8)
        codes[:, ::48] = torch.randint(0, 16, (rows, K // 48), generator=r, dtype=torch.uint8)
        s = torch.randint(scale - 3, scale + 1, (K // 32, rows), generator=r, dtype=torch.uint8)
        v = levels[codes.long()] * torch.exp2(s.double() - 127).T.repeat_interleave(32, dim=1)
        pitched = torch.zeros((K // 32, (rows + 15) // 16 * 16), dtype=torch.uint8)
        pitched[:, :rows] = s
        return (codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda(), pitched.cuda()[:, :rows], v

    (aq, as_, a), (gq, gs, bg), (uq, us, bu) = make(M, 126), make(N, 127), make(N, 127)
    g, u = a @ bg.T, a @ bu.T
    if bn:
        binding.gemm_debug_force_tile(11, bn)
    d = binding.gemm_gated_e2m1(aq, as_, gq, gs, uq, us, act="relu")
    assert torch.equal(d.cpu(), (g.clamp(min=0) * u).float())  # G and U are exact
    near = (g.abs() <= 12).double()
    assert near.mean() > 0.5
    d = binding.gemm_gated_e2m1(aq, as_, gq, gs, uq, us, act=act)
    check(d.cpu() * near, act, g * near, u * near, (M, bn))


@pytest.mark.parametrize("act", ref.ACTS)
def test_backward_follows_the_forward_in_the_tail(act):
    """dU = dD act(G) rounded to float16 once: the activation's bound and half a unit of float16."""
    g = torch.linspace(-9, 9, 20000).half()
    G = g.repeat(8, 1).cuda()
    dD = (2.0 ** torch.arange(8, 16, dtype=torch.float64)).half()[:, None].expand(8, 20000).contiguous().cuda()
    zero = torch.zeros_like(G)
    *_, dU = binding.gemm_gated_backward(dD, G, zero, None, None, None, need_input=False, need_weights=False, act=act)
    g = G.cpu().double()
    want = dD.cpu().double() * ref.act64(act, g)
    fits = want.abs() < 65504  # (the largest products leave float16's range)
    e = want.abs() * bound(act, g)
    ref.assert_close(torch.where(fits.cuda(), dU, zero), torch.where(fits, want, torch.zeros_like(want)),
                     e + ref.rounding(want.abs() + e, OUT_F16), act)
