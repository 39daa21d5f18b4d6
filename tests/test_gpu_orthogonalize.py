"""gemm_orthogonalize on the GPU (needs a GB300) against the recurrence in 64 bits.

Bound, in the Frobenius norm |.| (|.|2: the largest singular value): a step from X, with P = X X^T
over l and Q = b P + c P^2 over s, whose operands are rounded by at most h of themselves (2^-11, one
float16; 2^-22, two; half a unit of the subnormal range, 2^-25, an element before the scaling by
2^12), makes these errors:
    eP = (2 h + h^2 + sum(l)) |X|^2 + (2^-23 + h) |P| + s 2^-37
    eQ = (|b| + 2 |c| (|P|2 + eP)) eP + sum(s) |c| (|P| + eP)^2 + 2^-22 (|b| |P| + |c| |P|2 |P|) + h |Q| + s 2^-37
    eX = eQ |X|2 (1 + h) + (|Q|2 h + sum(s) (|Q| + eQ)) |X| + 2^-22 (|a| |X| + |Q| |X|2) + r |X'| + sqrt(m n) 2^-37
(r: 2^-22, the iterate's two parts, or in the last step the rounding to Y) and passes an error e of
X on as L e, L the largest slope of a x + b x^3 + c x^5 up to the largest singular value (and e
itself): the divided differences of a function are at most its largest slope.  sum(K) is gated_ref's
bound of a tensor-core sum.
"""
import numpy as np
import pytest
import torch

import gated_ref as ref
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding

pytestmark = pytest.mark.gpu

FORMS = {"auto": (0, 0), "single64": (1, 64), "single128": (1, 128), "pair256": (3, 256)}
MUON = (3.4445, -4.7750, 2.0315)
QUINTIC = (1.875, -1.25, 0.375)  # slope at most 1.875: errors stay small over many steps
EPS = 1e-7
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK


def recurrence(x, coefs, steps, eps, out):
    """(Y, bound of |error|) of one matrix in 64 bits."""
    a, b, c = coefs
    x = x.double().cpu()
    x = x / (x.norm() + eps)
    if x.shape[0] > x.shape[1]:
        x = x.T
        flip = True
    else:
        flip = False
    s, l = x.shape
    two = lambda m: torch.linalg.matrix_norm(m, 2).item()  # noqa: E731
    # the norm: float32 sums of N squares (2^-24 each, pairwise in part: at most the chain of a
    # thread), the root, the division and a product; then the iterate's two parts
    e = 2.0 ** -16 * x.norm().item() + (s * l) ** 0.5 * 2.0 ** -37
    more = 2 if s < 256 else 0
    exact = {torch.float32: steps, torch.float16: 1 + more, torch.bfloat16: more}[out]
    for i in range(steps):
        h = 2.0 ** -22 if i >= steps - exact else 2.0 ** -11
        p = x @ x.T
        q = b * p + c * (p @ p)
        y = a * x + q @ x
        X, P, Q, Y = (m.norm().item() for m in (x, p, q, y))
        X2, P2, Q2 = two(x) + e, two(p), two(q)
        grid = np.linspace(0.0, X2, 2001)
        L = np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max() + 1e-3 * (abs(a) + abs(b) + abs(c))
        eP = (2 * h + h * h + ref.sum_bound(l)) * X * X + (2.0 ** -23 + h) * P + s * 2.0 ** -37
        eQ = ((abs(b) + 2 * abs(c) * (P2 + eP)) * eP + ref.sum_bound(s) * abs(c) * (P + eP) ** 2
              + 2.0 ** -22 * (abs(b) * P + abs(c) * P2 * P) + h * Q + s * 2.0 ** -37)
        last = HALF[out] if i == steps - 1 else 2.0 ** -22
        eX = (eQ * X2 * (1 + h) + (Q2 * h + ref.sum_bound(s) * (Q + eQ)) * X
              + 2.0 ** -22 * (abs(a) * X + Q * X2) + last * Y
              + (s * l) ** 0.5 * (2.0 ** -25 if out == torch.float16 and i == steps - 1 else 2.0 ** -37))
        e = L * e + eX
        x = y
    return (x.T if flip else x), e


def stack(count, m, n, dtype, seed, scale=1.0, pad=3):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((count, m, n), generator=gen) + 3 * torch.randn((count, m, 1), generator=gen) * torch.randn((count, 1, n), generator=gen)
    buf = torch.full((count, m + 1, n + pad), float("nan"))
    buf[:, :m, :n] = x * scale
    return buf.to(dtype).cuda()[:, :m, :n]


def check(X, coefs, steps, out=None, eps=EPS, Y=None):
    out = X.dtype if out is None else out
    if Y is None:
        Y = torch.empty(X.shape, dtype=out, device="cuda")
    inputs = X.clone()
    binding.gemm_orthogonalize(X, Y, steps=steps, coefs=coefs, eps=eps)
    for i in range(X.shape[0]):
        want, bound = recurrence(inputs[i], coefs, steps, eps, out)
        err = (Y[i].cpu().double() - want).norm().item()
        assert err <= bound, (tuple(X.shape), X.dtype, out, coefs, steps, i, err, bound)
    return Y


SIZES = [(1, 1, 1), (1, 1, 40), (2, 40, 1), (3, 64, 64), (2, 65, 130), (2, 130, 63), (1, 129, 257), (1, 300, 200),
         (2, 200, 520), (1, 513, 515)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("count,m,n", SIZES)
def test_one_step(form, count, m, n):
    binding.gemm_debug_force_tile(*FORMS[form])
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)):
        check(stack(count, m, n, dtype, m + n), MUON, 1, out)


@pytest.mark.parametrize("count,m,n", [(2, 64, 200), (1, 200, 64), (2, 130, 257), (1, 600, 520), (1, 1000, 1367)])
def test_five_steps(count, m, n):
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        check(stack(count, m, n, dtype, m), QUINTIC, 5)
        check(stack(count, m, n, dtype, m), MUON, 2)
    check(stack(count, m, n, torch.float32, m), MUON, 5)


def test_singular_values_reach_one():
    """Ten steps of the convergent polynomial on a matrix of singular values between 0.1 and 1 leave
    an orthogonal matrix: every step moves s towards 1, and 10 of them past 1 - 2^-11."""
    gen = torch.Generator().manual_seed(0)
    u, _ = torch.linalg.qr(torch.randn(96, 96, generator=gen, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(200, 96, generator=gen, dtype=torch.float64))
    x = (u * torch.linspace(0.1, 1.0, 96, dtype=torch.float64)) @ v.T
    y = binding.gemm_orthogonalize(x.float().cuda(), steps=14, coefs=QUINTIC).cpu().double()
    exact = x.float().double()
    exact = exact / (exact.norm() + EPS)
    for _ in range(14):
        p = exact @ exact.T
        exact = QUINTIC[0] * exact + (QUINTIC[1] * p + QUINTIC[2] * (p @ p)) @ exact
    assert (torch.linalg.svdvals(exact) - 1).abs().max() < 2.0 ** -11
    # the steps' own errors are of the order of f16's rounding, and the polynomial's slope at 1 is 0
    assert (torch.linalg.svdvals(y) - 1).abs().max() < 16 * 2.0 ** -11


# Near orthogonal rows (P = I, a + b + c = 1, slope 0) the last step alone moves a singular value: what P's sum
# drops, at most sum_bound(l) of its diagonal, by |b + 2 c|; what P P's and the update's drop, sum_bound(s), by c
# and |b + c|; the operands' 22 bits and the last rounding, 2^-22 each, at most six times together.  For QUINTIC
# and 96 x 200: 5.5e-6; errors of no common sign across a row average out, the rest of 1e-5 is for them.
SINGULAR = 1e-5


def test_singular_values_follow_the_recurrence():
    """A float32 result's singular values against those of the recurrence in 64 bits: with the products X X^T and
    b P + c P^2 in one float16 they are off by 2e-4 (test_orthogonalize_bounds.py plants that)."""
    x = spread_matrix()
    want = torch.linalg.svdvals(recurrence(x, QUINTIC, 14, EPS, torch.float32)[0])
    y = binding.gemm_orthogonalize(x.cuda(), steps=14, coefs=QUINTIC).cpu().double()
    assert (torch.linalg.svdvals(y) - want).abs().max() < SINGULAR


def spread_matrix():
    """96 x 200 with singular values from 0.1 to 1."""
    gen = torch.Generator().manual_seed(0)
    u, _ = torch.linalg.qr(torch.randn(96, 96, generator=gen, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(200, 96, generator=gen, dtype=torch.float64))
    return ((u * torch.linspace(0.1, 1.0, 96, dtype=torch.float64)) @ v.T).float()


@pytest.mark.parametrize("scale", [1e-12, 1e-3, 1.0, 1e6])
def test_scales(scale):
    """The norm is divided out: small and large matrices alike."""
    check(stack(2, 70, 150, torch.float32, 1, scale), MUON, 1, eps=0.0)
    check(stack(2, 150, 70, torch.bfloat16, 1, scale), QUINTIC, 2, eps=0.0)


def test_in_place_and_strided():
    X = stack(3, 90, 70, torch.bfloat16, 4)
    want = binding.gemm_orthogonalize(X, steps=3)
    Y = stack(3, 90, 70, torch.bfloat16, 5, pad=11)
    binding.gemm_orthogonalize(X, Y, steps=3)
    assert torch.equal(Y, want)
    binding.gemm_orthogonalize(X, X, steps=3)
    assert torch.equal(X, want)
    assert torch.equal(binding.gemm_orthogonalize(stack(3, 90, 70, torch.bfloat16, 4)[1], steps=3), want[1])


def test_padding_is_left_alone():
    X = stack(2, 60, 45, torch.float32, 4)
    buf = torch.full((2, 61, 51), 7.0, device="cuda")
    binding.gemm_orthogonalize(X, buf[:, :60, :45])
    assert (buf[:, 60:] == 7).all() and (buf[:, :, 45:] == 7).all()
    assert torch.isfinite(buf[:, :60, :45]).all()


@pytest.mark.parametrize("n", [33, 34, 66, 67, 98, 129, 130, 259])
def test_row_ends_between_words(n):
    X = stack(2, 70, n, torch.float32, n)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        buf = torch.full((2, 71, n + 3 - n % 2), 7.0, dtype=out, device="cuda")
        check(X, MUON, 2, out, Y=buf[:, :70, :n])
        assert (buf[:, 70:] == 7).all() and (buf[:, :, n:] == 7).all()
        assert torch.equal(buf[:, :70, :n], binding.gemm_orthogonalize(X, torch.empty((2, 70, n + 8 - n % 8), dtype=out, device="cuda")[:, :, :n], steps=2))


def test_zeros_and_what_is_not_finite():
    X = stack(4, 50, 80, torch.float32, 6)
    good = binding.gemm_orthogonalize(X)
    X[0] = 0
    X[2, 3, 3] = float("inf")
    X[3, 49, 79] = float("nan")
    Y = binding.gemm_orthogonalize(X)
    assert (Y[0] == 0).all()
    assert torch.equal(Y[1], good[1])
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[3]).all()
    assert torch.isnan(binding.gemm_orthogonalize(torch.zeros(4, 4, device="cuda"), eps=0.0)).all()


@pytest.mark.parametrize("eps", [1e-30, 1e-36, 1e-44])
@pytest.mark.parametrize("m,n", [(50, 80), (300, 200), (16, 1000), (130, 3000)])
def test_zeros_whatever_eps(m, n, eps):
    """A matrix of zeros gives zeros for every eps above 0, one whose reciprocal is no float32 number
    among them; its neighbours, whose norm such an eps does not change, are what they are without."""
    X = stack(3, m, n, torch.float32, 6)
    good = binding.gemm_orthogonalize(X, eps=0.0)
    X[1] = 0
    Y = binding.gemm_orthogonalize(X, eps=eps)
    assert (Y[1] == 0).all()
    assert torch.equal(Y[0], good[0]) and torch.equal(Y[2], good[2])
    assert torch.isnan(binding.gemm_orthogonalize(X, eps=0.0)[1]).all()


@pytest.mark.parametrize("count,m,n", [(2, 448, 449), (1, 449, 512), (2, 512, 448), (1, 513, 449)])
def test_sums_at_the_length_that_two_ctas_share(count, m, n):
    """Seven, eight and nine blocks of 64: sums of eight and more are shared where that form is forced."""
    binding.gemm_debug_force_tile(3, 256)
    check(stack(count, m, n, torch.float32, m + n), MUON, 1)
    check(stack(count, m, n, torch.bfloat16, m + n), MUON, 2, torch.float32)


def test_iterates_past_their_range():
    """An element of 16 and more between the steps is not finite in Y; the other matrices of the stack
    are not concerned, nor is the last step's result."""
    X = stack(3, 300, 200, torch.float32, 6)
    good = binding.gemm_orthogonalize(X, steps=2)
    X[1] = 0
    X[1, 7, 9] = 5.0
    Y = binding.gemm_orthogonalize(X, steps=2, coefs=(1.0, -0.5, 0.0))
    assert torch.isfinite(Y).all()
    assert not torch.isfinite(binding.gemm_orthogonalize(X, steps=2, coefs=(20.0, -0.5, 0.0))[1, 7, 9])
    one = binding.gemm_orthogonalize(X, steps=1, coefs=(20.0, -0.5, 0.0))
    assert abs(one[1, 7, 9].item() - 19.5) < 1e-4
    assert torch.equal(binding.gemm_orthogonalize(X, steps=2)[::2], good[::2])


def test_same_bits_every_time():
    X = stack(5, 300, 200, torch.bfloat16, 8)
    a = binding.gemm_orthogonalize(X)
    for _ in range(3):
        assert torch.equal(binding.gemm_orthogonalize(X), a)


def test_a_stack_larger_than_the_workspace():
    """Taken in parts: each matrix as if alone."""
    X = torch.randn((20000, 96, 100), device="cuda").bfloat16()
    Y = binding.gemm_orthogonalize(X, steps=2)
    for i in (0, 1, 9999, 13000, 19999):
        assert torch.equal(Y[i], binding.gemm_orthogonalize(X[i], steps=2)), i


def test_elements_past_32_bits():
    """Matrices so far apart that element numbers do not fit 32 bits."""
    X, far = stack(3, 90, 70, torch.bfloat16, 4), (1 << 31) + 5
    big = torch.empty(2 * far + 90 * 70, dtype=torch.bfloat16, device="cuda").as_strided((3, 90, 70), (far, 70, 1))
    big.copy_(X)
    want = binding.gemm_orthogonalize(X, steps=2)
    assert torch.equal(binding.gemm_orthogonalize(big, steps=2), want)
    binding.gemm_orthogonalize(X, big, steps=2)
    assert torch.equal(big, want)


def test_single_rows_far_apart():
    """Matrices of one row, further apart than the largest pitch."""
    X, far = stack(3, 1, 70, torch.bfloat16, 4), (1 << 31) + 8
    big = torch.empty(2 * far + 70, dtype=torch.bfloat16, device="cuda").as_strided((3, 1, 70), (far, far, 1))
    for form in ((0, 0), (1, 64)):
        binding.gemm_debug_force_tile(*form)
        want = binding.gemm_orthogonalize(X, steps=2)
        big.copy_(X)
        assert torch.equal(binding.gemm_orthogonalize(big, steps=2), want)
        binding.gemm_orthogonalize(X, big, steps=2)
        assert torch.equal(big, want)


@pytest.mark.parametrize("form", [(1, 64), (1, 128), (3, 256), (0, 0)])
@pytest.mark.parametrize("count,m,n", [(3, 700, 900), (2, 1100, 380), (1, 2000, 1030)])
def test_more_tiles_than_ctas_hold(form, count, m, n):
    binding.gemm_debug_force_tile(*form)
    check(stack(count, m, n, torch.float32, m + n), MUON, 2)


@pytest.mark.parametrize("count,m,n", [(1, 41, 3000), (1, 3001, 41), (2, 2500, 130), (1, 260, 5000), (3, 64, 2117), (1, 6000, 1),
                                       (1, 257, 2600), (5, 4096, 16)])
def test_long_sums_of_few_tiles(count, m, n):
    """The sums of X X^T (X^T X) in parts, which a kernel of its own adds."""
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)):
        check(stack(count, m, n, dtype, m + n), MUON, 1, out)
        check(stack(count, m, n, dtype, m + n), QUINTIC, 4, out)
    X = stack(count, m, n, torch.bfloat16, 3)
    assert torch.equal(binding.gemm_orthogonalize(X), binding.gemm_orthogonalize(X))


SMALL = [(1, 16, 4096), (1, 4096, 16), (2, 64, 1000), (2, 1001, 63), (200, 16, 64), (30, 33, 17), (1, 5, 9), (3, 61, 61), (20, 1, 300),
         (1, 2, 2), (40, 40, 130)]


@pytest.mark.parametrize("count,m,n", SMALL)
def test_small_matrices(count, m, n):
    """One launch, in float32 throughout, which the bound of the two float16 parts covers: each of its
    roundings is 2^-24 of a value or of a term of a sum, of at most as many terms."""
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)):
        check(stack(count, m, n, dtype, m + n), MUON, 1, out)
        check(stack(count, m, n, dtype, m + n), QUINTIC, 5, out)
    X = stack(count, m, n, torch.float32, 3)
    Y = binding.gemm_orthogonalize(X)
    assert torch.equal(Y, binding.gemm_orthogonalize(X))
    buf = torch.full((count, m + 1, n + 5), 7.0, device="cuda")
    binding.gemm_orthogonalize(X, buf[:, :m, :n])
    assert torch.equal(buf[:, :m, :n], Y) and (buf[:, m:] == 7).all() and (buf[:, :, n:] == 7).all()
    binding.gemm_orthogonalize(X, X)
    assert torch.equal(X, Y)


@pytest.mark.parametrize("count,m,n", [(4, 16, 2000), (4, 300, 40), (30, 20, 30)])
def test_small_matrices_that_are_not_finite(count, m, n):
    X = stack(count, m, n, torch.float32, 6)
    good = binding.gemm_orthogonalize(X)
    X[0] = 0
    X[2, 3, 3] = float("inf")
    X[3, m - 1, n - 1] = float("nan")
    Y = binding.gemm_orthogonalize(X)
    assert (Y[0] == 0).all() and torch.equal(Y[1], good[1]) and torch.equal(Y[4:], good[4:])
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[3]).all()
    assert torch.isnan(binding.gemm_orthogonalize(torch.zeros(m, n, device="cuda"), eps=0.0)).all()


def test_small_matrices_captured_and_one_behind_another():
    X = stack(3, 24, 700, torch.bfloat16, 9)
    want = X
    for _ in range(3):
        want = binding.gemm_orthogonalize(want, steps=2)
    Y, s, graph = torch.empty_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        binding.gemm_orthogonalize(X, Y, steps=2)
        binding.gemm_orthogonalize(Y, Y, steps=2)
        binding.gemm_orthogonalize(Y, Y, steps=2)
    for _ in range(2):
        Y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
