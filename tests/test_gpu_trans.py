"""gemm_trans (operands stored K x M / K x N) on the GPU (needs a GB300): quarter-integers
compare bit for bit with 64-bit sums (every partial sum is exact in float32), normal
inputs within gated_ref's sum bound."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from gated_ref import assert_close, wide
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding
from tensor_core_gemm_02_gb300.workloads import OUT_BF16, OUT_F16, OUT_F32

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
STORED = [(False, True), (True, True), (True, False), (False, False)]
FORMS = {"auto": (0, 0), "single64": (1, 64), "single128": (1, 128), "single256": (1, 256),
         "pair256": (3, 256), "pair512": (4, 512)}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK


def operands(seed, M, N, K, ta, tb, dtype, exact):
    r = torch.Generator().manual_seed(seed)
    A = wide(K if ta else M, M if ta else K, dtype, r, exact=exact)
    B = wide(K if tb else N, N if tb else K, dtype, r, exact=exact)
    return A, B, wide(M, N, torch.float32, r, exact=exact)


def product(A, B, ta, tb):
    a, b = A.cpu().double(), B.cpu().double()
    a, b = (a.T if ta else a), (b if tb else b.T)
    return a @ b, a.abs() @ b.abs()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("ta,tb", STORED[:3])
def test_exact_every_form(form, ta, tb):
    binding.gemm_debug_force_tile(*FORMS[form])
    for M, N, K in ((1, 1, 1), (128, 256, 64), (129, 70, 63), (300, 520, 65), (40, 1030, 328), (513, 515, 200)):
        for dtype, out in ((BF16, OUT_F32), (F16, OUT_BF16), (BF16, OUT_F16)):
            A, B, C = operands(M + N + K, M, N, K, ta, tb, dtype, True)
            s, _ = product(A, B, ta, tb)
            got = binding.gemm_trans(A, B, C, trans_a=ta, trans_b=tb, alpha=0.5, beta=2.0, out=out)
            want = (0.5 * s + 2.0 * C.cpu().double()).float().to(ref.out_dtype(out))
            assert torch.equal(got.cpu(), want), (form, M, N, K, dtype, out)
            got = binding.gemm_trans(A, B, trans_a=ta, trans_b=tb, out=out)
            assert torch.equal(got.cpu(), s.float().to(ref.out_dtype(out))), (form, M, N, K, dtype, out)


@pytest.mark.parametrize("form", ["auto", "skinny"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 130, 64), (3, 128, 1000), (16, 1030, 65), (17, 200, 2056),
                                   (33, 520, 4100), (64, 257, 328), (48, 4096, 1024)])
def test_exact_few_rows_of_a(form, M, N, K):
    """The swap-AB kernel with B stored K x N: partial tiles, K shared out over CTAs, ragged sizes."""
    binding.gemm_debug_force_tile(*((2, 0) if form == "skinny" else (0, 0)))
    for dtype, out in ((BF16, OUT_F32), (F16, OUT_BF16), (BF16, OUT_F16)):
        A, B, C = operands(M + N + K, M, N, K, False, True, dtype, True)
        s, _ = product(A, B, False, True)
        got = binding.gemm_trans(A, B, C, trans_b=True, alpha=0.5, beta=2.0, out=out)
        want = (0.5 * s + 2.0 * C.cpu().double()).float().to(ref.out_dtype(out))
        assert torch.equal(got.cpu(), want), (M, N, K, dtype, out)
        got = binding.gemm_trans(A, B, trans_b=True, out=out)
        assert torch.equal(got.cpu(), s.float().to(ref.out_dtype(out))), (M, N, K, dtype, out)


@pytest.mark.parametrize("ta,tb", STORED[:3])
@pytest.mark.parametrize("M,N,K", [(100, 130, 2056), (128, 64, 4096), (300, 257, 4100), (257, 1001, 8200),
                                   (66, 5, 3000)])
def test_exact_long_sums_in_parts(ta, tb, M, N, K):
    """Few tiles and many K blocks: the sum is cut into parts (the plan says how many), the parts
    added in a second kernel, with C (in place too), every output type and odd addresses."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert binding.gemm_query_plan(M, N, K, trans=(ta, tb), sm_count=sms).splits > 1
    for dtype, out in ((BF16, OUT_F32), (F16, OUT_BF16), (BF16, OUT_F16)):
        A, B, C = operands(M + N + K, M, N, K, ta, tb, dtype, True)
        s, _ = product(A, B, ta, tb)
        got = binding.gemm_trans(A, B, C, trans_a=ta, trans_b=tb, alpha=0.5, beta=2.0, out=out)
        want = (0.5 * s + 2.0 * C.cpu().double()).float().to(ref.out_dtype(out))
        assert torch.equal(got.cpu(), want), (dtype, out)
        buf = torch.full((M, N + 5), 9.0, dtype=ref.out_dtype(out), device="cuda")
        binding.gemm_trans(A, B, None, buf[:, 3:3 + N], trans_a=ta, trans_b=tb, out=out)
        assert torch.equal(buf[:, 3:3 + N].cpu(), s.float().to(ref.out_dtype(out))), (dtype, out)
        assert (buf[:, :3] == 9.0).all() and (buf[:, 3 + N:] == 9.0).all()
    acc = C.clone()
    binding.gemm_trans(A, B, acc, acc, trans_a=ta, trans_b=tb)
    assert torch.equal(acc.cpu(), (s + C.cpu().double()).float())


@pytest.mark.parametrize("ta,tb", STORED)
@pytest.mark.parametrize("M,N,K,dtype,out", [(1, 300, 4096, BF16, OUT_F32), (64, 4096, 1000, F16, OUT_F16),
                                             (500, 264, 4100, BF16, OUT_BF16)])
def test_random_within_bound(ta, tb, M, N, K, dtype, out):
    A, B, C = operands(K, M, N, K, ta, tb, dtype, False)
    s, t = product(A, B, ta, tb)
    d = 0.5 * s + C.cpu().double()
    e = 0.5 * ref.sum_bound(K) * t + (d.abs() + t) * 2.0 ** -23
    got = binding.gemm_trans(A, B, C, trans_a=ta, trans_b=tb, alpha=0.5, out=out)
    assert_close(got, d, e + ref.rounding(d.abs() + e, out), f"{ta} {tb}")


@pytest.mark.parametrize("ta,tb", STORED[:3])
def test_in_place_unaligned_and_k_zero(ta, tb):
    M, N, K = 70, 45, 96
    A, B, C = operands(3, M, N, K, ta, tb, F16, True)
    s, _ = product(A, B, ta, tb)
    want = (s + C.cpu().double()).float()
    acc = C.clone()
    binding.gemm_trans(A, B, acc, acc, trans_a=ta, trans_b=tb)  # accumulated onto D itself
    assert torch.equal(acc.cpu(), want)
    buf = torch.full((M, N + 5), 9.0, device="cuda")
    binding.gemm_trans(A, B, C, buf[:, 3:3 + N], trans_a=ta, trans_b=tb)  # D at an odd address
    assert torch.equal(buf[:, 3:3 + N].cpu(), want)
    assert (buf[:, :3] == 9.0).all() and (buf[:, 3 + N:] == 9.0).all()
    a0 = torch.empty((0, M) if ta else (M, 0), dtype=F16, device="cuda")
    b0 = torch.empty((0, N) if tb else (N, 0), dtype=F16, device="cuda")
    D = binding.gemm_trans(a0, b0, C, trans_a=ta, trans_b=tb, beta=0.5)
    assert torch.equal(D, 0.5 * C)
    assert (binding.gemm_trans(a0, b0, trans_a=ta, trans_b=tb) == 0).all()


def test_nan_stays_in_its_row():
    A, B, _ = operands(5, 200, 130, 264, True, True, BF16, True)
    clean = binding.gemm_trans(A, B, trans_a=True, trans_b=True)
    A[9, 4] = float("nan")  # K row 9 of column 4: row 4 of D
    D = binding.gemm_trans(A, B, trans_a=True, trans_b=True)
    rows = torch.arange(200, device="cuda") != 4
    assert torch.isnan(D[4]).all() and torch.equal(D[rows], clean[rows])


@pytest.mark.parametrize("ta,tb", STORED[:3])
def test_timeout_reports_and_recovers(ta, tb):
    A, B, _ = operands(6, 300, 300, 512, ta, tb, BF16, True)
    good = binding.gemm_trans(A, B, trans_a=ta, trans_b=tb)
    assert device_status() == binding.GEMM_OK
    binding.gemm_set_wait_timeout(50_000_000)
    binding.gemm_debug_inject(1)
    try:
        binding.gemm_trans(A, B, trans_a=ta, trans_b=tb)
        assert device_status() == binding.GEMM_ERR_TIMEOUT
    finally:
        binding.gemm_debug_inject(0)
        binding.gemm_set_wait_timeout(0)
    assert torch.equal(binding.gemm_trans(A, B, trans_a=ta, trans_b=tb), good)


def test_linear_layer_gradients_match_the_stored_transposes():
    """dX = dY W and dW = dY^T X read in place equal the plain products of transposed copies."""
    r = torch.Generator().manual_seed(1)
    X, W, dY = (wide(m, n, BF16, r, exact=True) for m, n in ((200, 136), (264, 136), (200, 264)))
    dX = binding.gemm_trans(dY, W, trans_b=True)
    dW = binding.gemm_trans(dY, X, trans_a=True, trans_b=True)
    assert torch.equal(dX, binding.gemm_bf16(dY, W.T.contiguous()))
    assert torch.equal(dW, binding.gemm_bf16(dY.T.contiguous(), X.T.contiguous()))
    assert np.isfinite(dW.cpu().numpy()).all()


@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16, OUT_F16])
@pytest.mark.parametrize("ta,tb", STORED[:3])
def test_output_rows_not_16_bytes_apart(ta, tb, out):
    """D written without TMA, with and without C, on every form: the same bits as an aligned D,
    nothing beside it."""
    M, N, K = 300, 205, 200
    dtype = {OUT_F32: torch.float32, OUT_BF16: BF16, OUT_F16: F16}[out]
    A, B, C = operands(3, M, N, K, ta, tb, BF16, False)
    for name, form in FORMS.items():
        for c in (None, C):
            binding.gemm_debug_force_tile(*form)
            aligned = torch.empty((M, 208), dtype=dtype, device="cuda")[:, :N]
            binding.gemm_trans(A, B, c, aligned, trans_a=ta, trans_b=tb, alpha=0.5, beta=2.0, out=out)
            buf = torch.full((M + 1, 211), float("nan"), dtype=dtype, device="cuda")
            D = buf[:M, 3:3 + N]
            binding.gemm_trans(A, B, c, D, trans_a=ta, trans_b=tb, alpha=0.5, beta=2.0, out=out)
            assert torch.equal(D, aligned), (name, c is not None)
            assert int(torch.isnan(buf).sum()) == buf.numel() - M * N


@pytest.mark.parametrize("ta,tb", STORED[:3])
def test_exact_sums_in_parts_on_pairs(ta, tb):
    """More rows than one block and a long sum: parts on CTA pairs, with C and at an odd address."""
    M, N, K = 500, 1000, 8200
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = binding.gemm_query_plan(M, N, K, trans=(ta, tb), sm_count=sms)
    assert plan.splits > 1 and (sms != 152 or plan.kernel == 3)
    A, B, C = operands(11, M, N, K, ta, tb, BF16, True)
    s, _ = product(A, B, ta, tb)
    got = binding.gemm_trans(A, B, C, trans_a=ta, trans_b=tb, alpha=0.5, beta=2.0, out=OUT_F16)
    assert torch.equal(got.cpu(), (0.5 * s + 2.0 * C.cpu().double()).float().half())
    buf = torch.full((M, N + 5), 9.0, device="cuda")
    binding.gemm_trans(A, B, None, buf[:, 3:3 + N], trans_a=ta, trans_b=tb)
    assert torch.equal(buf[:, 3:3 + N].cpu(), s.float())
    assert (buf[:, :3] == 9.0).all() and (buf[:, 3 + N:] == 9.0).all()
