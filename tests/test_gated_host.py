"""Host-side checks of the gated entry points that need no GPU: refusals before any CUDA call,
the binding's own checks, and plans."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import gated_ref as ref
from tensor_core_gemm_02_gb300 import binding
from tensor_core_gemm_02_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load_library()


# Fake, never-dereferenced device addresses, far apart: every refusal comes before any CUDA call.
def at(i):
    return 0x10000000 * (i + 1)


GATED = dict(M=64, N=64, K=64, bf16=1, A=at(0), lda=64, Bg=at(1), ldbg=64, Bu=at(2), ldbu=64, G=None, ldg=0,
             U=None, ldu=0, D=at(3), ldd=64, out=0, act=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(bf16=2), 1), (dict(out=3), 1), (dict(act=-1), 1),
    (dict(act=5), 1), (dict(A=None), 1), (dict(Bg=None), 1), (dict(Bu=None), 1), (dict(D=None), 1),
    (dict(lda=63), 1), (dict(ldbg=56), 1), (dict(ldbu=56), 1), (dict(ldd=63), 1), (dict(G=at(4), ldg=63), 1),
    (dict(U=at(4), ldu=1), 1), (dict(A=at(0) + 8), 2), (dict(Bu=at(2) + 2), 2), (dict(lda=68), 2),
    (dict(ldbg=65), 2), (dict(D=at(3) + 2), 2), (dict(G=at(4) + 1, ldg=64), 2), (dict(M=1 << 31), 3),
    (dict(ldd=1 << 31), 3), (dict(D=at(0) + 128), 4), (dict(D=at(2)), 4), (dict(G=at(3) + 64, ldg=64), 4),
    (dict(G=at(4), ldg=64, U=at(4), ldu=64), 4), (dict(U=at(1) + 16, ldu=64), 4),
    (dict(M=0, A=None), 0), (dict(N=0), 0),
])
def test_gated_refusals(lib, kw, code):
    a = dict(GATED, **kw)
    assert lib.gemm_gated(*a.values(), None) == code


FP4 = dict(M=64, N=64, K=64, Aq=at(0), ldaq=32, As=at(1), ldas=64, Bgq=at(2), ldbgq=32, Bgs=at(3), ldbgs=64,
           Buq=at(4), ldbuq=32, Bus=at(5), ldbus=64, D=at(6), ldd=64, out=0, act=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(out=7), 1), (dict(act=9), 1), (dict(K=48), 3), (dict(K=1 << 31), 3),
    (dict(Aq=None), 1), (dict(As=None), 1), (dict(Bgs=None), 1), (dict(Buq=None), 1), (dict(ldaq=16), 1),
    (dict(ldas=63), 1), (dict(ldbus=10), 1), (dict(Aq=at(0) + 8), 2), (dict(ldbuq=40), 2), (dict(D=at(6) + 1), 2),
    (dict(D=at(3)), 4), (dict(D=at(1) + 63), 2), (dict(D=at(5) + 64), 4), (dict(D=at(2) + 32), 4), (dict(M=0), 0),
])
def test_gated_e2m1_refusals(lib, kw, code):
    assert lib.gemm_gated_e2m1(*dict(FP4, **kw).values(), None) == code


BACK = dict(M=64, N=64, K=64, bf16=1, dD=at(0), lddd=64, G=at(1), ldg=64, U=at(2), ldu=64, A=at(3), lda=64,
            Bg=at(4), ldbg=64, Bu=at(5), ldbu=64, dG=at(6), lddg=64, dU=at(7), lddu=64, dA=at(8), ldda=64,
            dBg=at(9), lddbg=64, dBu=at(10), lddbu=64, out=0, act=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(bf16=3), 1), (dict(out=-1), 1), (dict(act=6), 1), (dict(dD=None), 1), (dict(G=None), 1),
    (dict(U=None), 1), (dict(A=None), 1), (dict(Bg=None), 1), (dict(dG=None), 1), (dict(dU=None), 1),
    (dict(dBg=None), 1), (dict(dBu=None), 1), (dict(lddd=10), 1), (dict(ldda=8), 1), (dict(lddbu=63), 1),
    (dict(dG=at(6) + 8), 2), (dict(lddu=68), 2), (dict(A=at(3) + 2), 2), (dict(ldbg=66), 2), (dict(G=at(1) + 1), 2),
    (dict(dA=at(8) + 2), 2), (dict(N=1 << 31), 3), (dict(lddbg=1 << 31), 3), (dict(dG=at(0)), 4),
    (dict(dG=at(2)), 4), (dict(dU=at(1)), 4), (dict(dG=at(1) + 16), 4), (dict(dG=at(1), lddg=72), 4),
    (dict(dU=at(6)), 4), (dict(dA=at(3)), 4), (dict(dBg=at(4)), 4), (dict(dBu=at(9) + 256), 4), (dict(dA=at(1)), 4),
    (dict(dBu=at(0)), 4),
])
def test_gated_backward_refusals(lib, kw, code):
    assert lib.gemm_gated_backward(*dict(BACK, **kw).values(), None) == code


TRANS = dict(M=64, N=32, K=128, bf16=1, ta=1, A=at(0), lda=64, tb=1, B=at(1), ldb=32, C=None, ldc=0, D=at(2), ldd=32,
             out=0, alpha=1.0, beta=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(bf16=2), 1), (dict(ta=2), 1), (dict(tb=-1), 1), (dict(out=4), 1), (dict(A=None), 1),
    (dict(B=None), 1), (dict(D=None), 1), (dict(lda=56), 1), (dict(ldb=24), 1), (dict(ta=0), 1), (dict(tb=0), 1),
    (dict(ldd=31), 1), (dict(C=at(3), ldc=31), 1), (dict(lda=66), 2), (dict(B=at(1) + 4), 2), (dict(D=at(2) + 2), 2),
    (dict(C=at(3) + 1, ldc=32), 2), (dict(K=1 << 31), 3), (dict(ldb=1 << 31), 3), (dict(D=at(0) + 127 * 128), 4),
    (dict(D=at(1)), 4), (dict(C=at(2) + 4, ldc=32), 4), (dict(C=at(2), ldc=40), 4), (dict(C=at(2), ldc=32, out=1), 4),
    (dict(M=0), 0), (dict(N=0, B=None), 0),
])
def test_trans_refusals(lib, kw, code):
    assert lib.gemm_trans(*dict(TRANS, **kw).values(), None) == code


QUANT = dict(M=64, K=64, type=0, X=at(0), ldx=64, Q=at(1), ldq=32, S=at(2), lds=64, Y=None, ldy=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(type=3), 1), (dict(X=None), 1), (dict(Q=None), 1), (dict(S=None), 1), (dict(ldx=63), 1),
    (dict(ldq=16), 1), (dict(lds=63), 1), (dict(Y=at(3), ldy=10), 1), (dict(K=40), 3), (dict(M=1 << 31), 3),
    (dict(X=at(0) + 2), 2), (dict(Q=at(1) + 8), 2), (dict(ldq=40), 2), (dict(Y=at(3) + 1, ldy=64), 2),
    (dict(Q=at(0) + 16), 4), (dict(S=at(1) + 5), 4), (dict(Y=at(0), ldy=72), 4), (dict(Y=at(0) + 4, ldy=64), 4),
    (dict(S=at(0) + 1), 4), (dict(Y=at(2), ldy=64), 4), (dict(M=0, X=None), 0), (dict(K=0), 0),
])
def test_quantize_refusals(lib, kw, code):
    assert lib.gemm_quantize_e2m1(*dict(QUANT, **kw).values(), None) == code


def test_binding_refusals():
    h = lambda r, c, t=torch.float16: torch.zeros((r, c), dtype=t)  # noqa: E731
    with pytest.raises(TypeError):
        binding.gemm_gated(h(4, 8), h(4, 8, torch.bfloat16), h(4, 8))
    with pytest.raises(TypeError):
        binding.gemm_gated(h(4, 8), h(4, 8), h(4, 8), G=h(4, 4, torch.float32))
    with pytest.raises(ValueError):
        binding.gemm_gated(h(4, 8), h(4, 8), h(5, 8))
    with pytest.raises(ValueError):
        binding.gemm_gated(h(4, 8), h(4, 8), h(4, 8), act="swish")
    with pytest.raises(ValueError):
        binding.gemm_gated(h(4, 8), h(4, 8), h(4, 8), U=h(4, 8))
    with pytest.raises(ValueError):
        binding.gemm_gated_backward(h(4, 8), h(4, 8), h(4, 7), h(4, 8), h(8, 8), h(8, 8))
    with pytest.raises(TypeError):
        binding.gemm_gated_backward(h(4, 8, torch.float32), h(4, 8), h(4, 8), h(4, 8), h(8, 8), h(8, 8))
    with pytest.raises(ValueError):
        binding.gemm_trans(h(4, 8), h(4, 8), trans_a=True, trans_b=False)
    with pytest.raises(TypeError):
        binding.gemm_quantize_e2m1(torch.zeros((4, 32), dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.gemm_quantize_e2m1(h(4, 32), Q=torch.zeros((4, 15), dtype=torch.uint8))
    for call in (lambda: binding.gemm_gated(h(4, 8), h(4, 8), h(4, 8)),  # right, but not on a CUDA device
                 lambda: binding.gemm_trans(h(4, 8), h(8, 16), trans_b=True),
                 lambda: binding.gemm_gated_backward(h(4, 8), h(4, 8), h(4, 8), h(4, 16), h(8, 16), h(8, 16)),
                 lambda: binding.gemm_quantize_e2m1(h(4, 32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    u = lambda r, c: torch.zeros((r, c), dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):
        binding.gemm_gated_e2m1(u(4, 16), u(1, 4), u(8, 16), u(1, 8), u(8, 16), u(1, 7))


def test_plans(lib):
    plan = binding.gemm_query_plan
    assert plan(16, 14336, 4096, gated="16", sm_count=152).kernel == 2
    assert plan(16, 14336, 4096, gated="16", has_c=True, sm_count=152).kernel != 2  # products kept
    assert plan(65, 14336, 4096, gated="16", sm_count=152).kernel != 2
    assert plan(16, 14336, 0, gated="16", sm_count=152).kernel == 1
    p = plan(8192, 14336, 4096, gated="16", sm_count=152)
    assert (p.kernel, p.bn, p.tiles) == (3, 256, 32 * 112)
    assert plan(64, 1000, 4096, gated="e2m1", sm_count=152).kernel == 15
    assert plan(65, 1000, 4096, gated="e2m1", sm_count=152).kernel == 11
    assert plan(0, 8, 8, gated="16").kernel == 0 and plan(8, 0, 8, gated="e2m1").kernel == 0
    p = plan(4096, 14336, 8192, trans=(True, True), sm_count=152)
    assert (p.kernel, p.bn) == (4, 512)
    assert plan(100, 64, 0, trans=(False, True), sm_count=152).kernel == 1
    binding.gemm_debug_force_tile(3, 256)
    try:
        assert plan(16, 128, 64, gated="16").kernel == 3
        assert plan(16, 128, 64, trans=(True, False)).kernel == 3
        assert plan(16, 128, 0, gated="16").kernel == 1  # pairs need K > 0
    finally:
        binding.gemm_debug_force_tile(0, 0)


def test_reference_forms_agree_with_torch():
    """The tests' own 64-bit forms against torch's, and the quantiser's against exhaustive search."""
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    f = torch.nn.functional
    for name, fn in (("silu", f.silu), ("gelu", f.gelu), ("gelu_tanh", lambda x: f.gelu(x, approximate="tanh")),
                     ("relu", f.relu), ("sigmoid", torch.sigmoid)):
        assert torch.allclose(ref.act64(name, g), fn(g), rtol=1e-12, atol=1e-14)
        x = g.clone().requires_grad_()
        (slope,) = torch.autograd.grad(fn(x).sum(), x)
        assert torch.allclose(ref.slope64(name, g), slope, rtol=1e-11, atol=1e-13)
        assert slope.abs().max() <= ref.SLOPE[name]
    x = np.random.default_rng(0).normal(size=(4, 64)) * 3
    codes, scales, values = ref.quantize64(x)
    for i in range(4):
        for j in range(64):
            s = 2.0 ** (int(scales[i, j // 32]) - 127)
            assert abs(values[i, j] - x[i, j]) <= min(abs(np.sign(x[i, j]) * v * s - x[i, j]) for v in ref.LEVELS) + 1e-12
    assert (scales == np.floor(np.log2(np.abs(x).reshape(4, 2, 32).max(2))) + 125).all()


@pytest.mark.parametrize("has_c", [False, True])
@pytest.mark.parametrize("M,N,K", [(16, 4096, 4096), (512, 512, 8192), (8192, 8192, 512), (3, 5, 7)])
def test_plan_of_untransposed_operands_is_the_plain_one(lib, M, N, K, has_c):
    """gemm_trans with neither operand transposed runs gemm_f16 / gemm_bf16, and its plan says so."""
    fields = [name for name, _ in binding.Plan._fields_]
    plain = binding.gemm_query_plan(M, N, K, has_c=has_c, sm_count=152)
    got = binding.gemm_query_plan(M, N, K, has_c=has_c, sm_count=152, trans=(False, False))
    assert [getattr(got, f) for f in fields] == [getattr(plain, f) for f in fields]


def test_binding_without_torchs_private_calls():
    """The current device and stream come from torch's public calls where it lacks the private ones."""
    code = textwrap.dedent("""
        import types, torch
        for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
            if hasattr(torch._C, name):
                delattr(torch._C, name)
        torch.cuda.current_device = lambda: 1
        torch.cuda.current_stream = lambda device=None: types.SimpleNamespace(cuda_stream=100 + device)
        from tensor_core_gemm_02_gb300 import binding
        assert binding._stream_ptr(None) == 101 and binding._stream_ptr(7) == 7
        print("right")
        """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stdout + r.stderr
