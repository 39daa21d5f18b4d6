"""gemm_quantize_e2m1 on the GPU against the element-by-element definition (needs a GB300).
Every comparison is exact: scales and codes are integers, values powers of two times levels."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(autouse=True)
def _clean():
    assert device_status() == binding.GEMM_OK
    yield
    assert device_status() == binding.GEMM_OK


def check(X, **kw):
    Y = torch.full_like(X, 7.0)
    Q, S = binding.gemm_quantize_e2m1(X, Y=Y, **kw)
    codes, scales, values = ref.quantize64(X.float().cpu().numpy())
    assert np.array_equal(S.cpu().numpy(), scales.T)
    assert np.array_equal(Q.cpu().numpy(), ref.pack(codes))
    assert np.array_equal(Y.float().cpu().numpy(), values, equal_nan=True)
    Q2, S2 = binding.gemm_quantize_e2m1(X)  # without the values
    assert torch.equal(Q2, Q) and torch.equal(S2, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 14336), (3, 64), (16, 4096), (31, 288), (33, 256), (100, 800),
                                 (257, 1056)])
def test_rows_of_many_sizes(dtype, M, K):
    r = torch.Generator().manual_seed(M + K)
    X = torch.randn((M, K), generator=r) * torch.exp(torch.randn((M, 1), generator=r))
    X[M // 2, :32] = 0.0
    check(X.to(dtype).cuda())


@pytest.mark.parametrize("dtype", TYPES[1:])
def test_every_16_bit_value(dtype):
    """All 65536 patterns (NaNs and infinities included), sorted so that blocks hold neighbours,
    and shuffled so that they hold extremes."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).reshape(64, 1024)
    check(every.cuda())
    order = torch.randperm(65536, generator=torch.Generator().manual_seed(0))
    check(every.reshape(-1)[order].reshape(64, 1024).cuda())


def test_ties_signs_powers_and_extremes():
    block = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999999, 0.0, -0.0, 0.2499999,
                          0.2500001, 4.999999, 5.000001, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0,
                          -7.5, 1e-30, -1e-30, 0.5, 1.0, 2.0, 3.0])
    rows = [block * 2.0 ** e for e in (-149, -130, -127, -126, -125, -124, -100, -1, 0, 1, 60, 124, 125)]
    rows.append(torch.full((32,), 3.4028234e38))
    rows.append(torch.zeros(32))
    rows.append(-torch.zeros(32))
    rows.append(torch.full((32,), 2.0 ** -149))
    X = torch.stack(rows)
    X[X.abs() == float("inf")] = 1.0
    check(X.cuda())


def test_infinity_and_nan_make_their_block_nan():
    X = torch.randn((40, 128), generator=torch.Generator().manual_seed(2))
    X[3, 33], X[5, 0], X[39, 127] = float("inf"), float("nan"), float("-inf")
    for dtype in TYPES:
        check(X.to(dtype).cuda())
    Q, S = binding.gemm_quantize_e2m1(X.cuda())
    assert S[1, 3] == 255 and S[0, 5] == 255 and S[3, 39] == 255 and (S == 255).sum() == 3
    assert (Q[3, 16:32] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_strided_in_place_and_bounds(dtype):
    M, K = 37, 96
    r = torch.Generator().manual_seed(4)
    x = torch.randn((M, K), generator=r).to(dtype).cuda()
    codes, scales, values = ref.quantize64(x.float().cpu().numpy())
    buf = torch.full((M, K + 5), 9.0, dtype=dtype, device="cuda")
    X = buf[:, 1:1 + K]
    X.copy_(x)
    qb = torch.full((M, K // 2 + 16), 99, dtype=torch.uint8, device="cuda")
    sb = torch.full((K // 32 + 1, M + 3), 99, dtype=torch.uint8, device="cuda")
    binding.gemm_quantize_e2m1(X, qb[:, :K // 2], sb[:K // 32, 1:1 + M], Y=X)
    assert np.array_equal(X.float().cpu().numpy(), values) and (buf[:, 0] == 9).all() and (buf[:, 1 + K:] == 9).all()
    assert np.array_equal(qb[:, :K // 2].cpu().numpy(), ref.pack(codes)) and (qb[:, K // 2:] == 99).all()
    assert np.array_equal(sb[:K // 32, 1:1 + M].cpu().numpy(), scales.T)
    assert (sb[K // 32] == 99).all() and (sb[:, 0] == 99).all() and (sb[:, 1 + M:] == 99).all()


def test_empty_and_other_stream():
    for shape in ((0, 64), (5, 0)):
        Q, S = binding.gemm_quantize_e2m1(torch.empty(shape, device="cuda"))
        assert Q.shape == (shape[0], shape[1] // 2) and S.shape == (shape[1] // 32, shape[0])
    X = torch.randn((300, 512), generator=torch.Generator().manual_seed(8)).cuda()
    Q, S = binding.gemm_quantize_e2m1(X)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    Q2, S2 = torch.zeros_like(Q), torch.zeros_like(S)
    s.wait_stream(torch.cuda.current_stream())
    binding.gemm_quantize_e2m1(X, Q2, S2, stream=s)
    s.synchronize()
    assert torch.equal(Q, Q2) and torch.equal(S, S2)


def test_product_of_quantised_operands():
    """gemm_e2m1 on quantised rows equals the product of the values they stand for (16-level values
    of like scales: sums exact in float32)."""
    r = torch.Generator().manual_seed(6)
    A, B = ((torch.randint(-6, 7, (n, 256), generator=r).float()).cuda() for n in (130, 70))
    va, vb = torch.empty_like(A), torch.empty_like(B)
    D = binding.gemm_e2m1(*binding.gemm_quantize_e2m1(A, Y=va), *binding.gemm_quantize_e2m1(B, Y=vb))
    assert torch.equal(D.cpu().double(), va.cpu().double() @ vb.cpu().double().T)
