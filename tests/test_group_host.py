"""Host-side checks of the entry points for groups that need no GPU: refusals before any CUDA call
and the binding's own checks."""
import pytest
import torch

from tensor_core_gemm_02_gb300 import binding
from tensor_core_gemm_02_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load_library()


# Fake, never-dereferenced device addresses, far apart: every refusal comes before any CUDA call.
def at(i):
    return 0x10000000 * (i + 1)


ROWS = dict(M=64, groups=8, choices=2, ids=at(0), offsets=at(1), order=at(2), rows=at(3))


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(groups=-1), 1), (dict(choices=0), 1), (dict(ids=None), 1), (dict(offsets=None), 1),
    (dict(order=None), 1), (dict(M=1 << 31), 3), (dict(groups=1025), 3), (dict(choices=1 << 31), 3),
    (dict(ids=at(0) + 2), 2), (dict(offsets=at(1) + 1), 2), (dict(order=at(2) + 3), 2), (dict(rows=at(3) + 2), 2),
    (dict(order=at(0) + 252), 4), (dict(offsets=at(0)), 4), (dict(offsets=at(2) + 252), 4), (dict(rows=at(2)), 4),
    (dict(rows=at(0) + 4), 4),
])
def test_group_rows_refusals(lib, kw, code):
    assert lib.gemm_group_rows(*dict(ROWS, **kw).values(), None) == code


GROUPED = dict(M=64, N=32, K=128, groups=4, bf16=1, A=at(0), a_rows=0, lda=128, idx=None, offsets=at(1), tb=0, B=at(2),
               ldb=128, stride_b=4096, D=at(3), ldd=32, out=0, alpha=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(groups=-1), 1), (dict(bf16=2), 1), (dict(tb=2), 1),
    (dict(out=3), 1), (dict(A=None), 1), (dict(B=None), 1), (dict(D=None), 1), (dict(offsets=None), 1),
    (dict(lda=120), 1), (dict(ldb=120), 1), (dict(ldd=31), 1), (dict(stride_b=4088), 1), (dict(stride_b=0), 1),
    (dict(tb=1, ldb=24), 1), (dict(tb=1, ldb=32, stride_b=4000), 1), (dict(idx=at(4)), 1),
    (dict(idx=at(4), a_rows=-3), 1),
    (dict(A=at(0) + 8), 2), (dict(lda=132), 2), (dict(B=at(2) + 2), 2), (dict(ldb=130, stride_b=8192), 2),
    (dict(stride_b=4100), 2), (dict(D=at(3) + 2), 2), (dict(offsets=at(1) + 2), 2), (dict(idx=at(4) + 1, a_rows=9), 2),
    (dict(M=1 << 31), 3), (dict(groups=1025), 3), (dict(ldd=1 << 31), 3), (dict(idx=at(4), a_rows=1 << 31), 3),
    (dict(N=1 << 30, groups=1000, ldd=1 << 30, stride_b=1 << 37), 3), (dict(stride_b=1 << 62), 3),
    (dict(D=at(0) + 64), 4), (dict(D=at(2) + 8), 4), (dict(D=at(2) + 4 * 4096 * 2 - 16), 4), (dict(D=at(1)), 4),
    (dict(D=at(4), idx=at(4) + 64, a_rows=4), 4),
    (dict(M=0, A=None), 0), (dict(N=0, B=None), 0), (dict(groups=0, B=None, offsets=None), 0),
])
def test_grouped_refusals(lib, kw, code):
    assert lib.gemm_grouped(*dict(GROUPED, **kw).values(), None) == code


WEIGHTS = dict(M=64, N=32, K=128, groups=4, bf16=0, dD=at(0), lddd=32, A=at(1), lda=128, offsets=at(2), dB=at(3),
               lddb=128, stride_db=4096, out=0, alpha=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(bf16=-1), 1), (dict(out=5), 1), (dict(dD=None), 1), (dict(A=None), 1), (dict(dB=None), 1),
    (dict(offsets=None), 1), (dict(lddd=24), 1), (dict(lda=120), 1), (dict(lddb=127), 1), (dict(stride_db=4095), 1),
    (dict(dD=at(0) + 4), 2), (dict(lda=130), 2), (dict(dB=at(3) + 1), 2), (dict(offsets=at(2) + 2), 2),
    (dict(K=1 << 31), 3), (dict(groups=2000), 3), (dict(lddb=1 << 31, stride_db=1 << 40), 3),
    (dict(dB=at(0)), 4), (dict(dB=at(1) + 64), 4), (dict(dB=at(2) + 16), 4),
    (dict(N=0, dD=None), 0), (dict(K=0), 0), (dict(groups=0, dB=None), 0),
])
def test_weights_refusals(lib, kw, code):
    assert lib.gemm_grouped_weights(*dict(WEIGHTS, **kw).values(), None) == code


ORTHO = dict(count=3, M=64, N=32, type=1, X=at(0), ldx=32, stride_x=2048, out=0, Y=at(1), ldy=32, stride_y=2048,
             steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(M=-1), 1), (dict(type=3), 1), (dict(out=-1), 1), (dict(steps=0), 1),
    (dict(steps=101), 1), (dict(a=float("nan")), 1), (dict(c=float("inf")), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(X=None), 1), (dict(Y=None), 1), (dict(ldx=31), 1), (dict(ldy=16), 1),
    (dict(stride_x=2047), 1), (dict(stride_y=100), 1), (dict(X=at(0) + 1), 2), (dict(Y=at(1) + 2), 2),
    (dict(M=1 << 31), 3), (dict(ldx=1 << 31, stride_x=1 << 40), 3),
    (dict(M=1 << 30, N=1 << 20, ldx=1 << 20, ldy=1 << 20, count=1), 3),
    (dict(Y=at(0)), 4), (dict(Y=at(0), out=1, stride_y=2056), 4), (dict(Y=at(0) + 64, out=1), 4),
    (dict(count=0, X=None), 0), (dict(M=0), 0), (dict(N=0, Y=None), 0),
])
def test_orthogonalize_refusals(lib, kw, code):
    assert lib.gemm_orthogonalize(*dict(ORTHO, **kw).values(), None) == code


def test_binding_refusals():
    z = torch.zeros
    h = dict(dtype=torch.bfloat16)
    off = z(4, dtype=torch.int32)
    for args, kw, err in (
            ((z(4, 8), z(3, 8, 8), off), {}, TypeError),
            ((z(4, 8, **h), z(3, 8, 8), off), {}, TypeError),
            ((z(4, 8, **h), z(3, 8, 9, **h), off), {}, ValueError),
            ((z(4, 8, **h), z(3, 9, 8, **h), off), dict(trans_b=True), ValueError),
            ((z(4, 8, **h), z(2, 8, 8, **h), off), {}, ValueError),
            ((z(4, 8, **h), z(3, 8, 8, **h), off.long()), {}, TypeError),
            ((z(4, 8, **h), z(3, 8, 8, **h), z(8, dtype=torch.int32)[::2]), {}, ValueError),
            ((z(4, 8, **h), z(3, 8, 8, **h), off), dict(idx=z(4, dtype=torch.int64)), TypeError),
            ((z(4, 8, **h), z(3, 8, 8, **h), off, z(4, 9)), {}, ValueError),
            ((z(4, 8, **h), z(3, 8, 8, **h), off, z(4, 8, **h)), {}, TypeError),
            ((z(4, 16, **h)[:, ::2], z(3, 8, 8, **h), off), {}, ValueError),
            ((z(4, 8, **h), z(3, 8, 8, **h), off, z(4, 8)), {}, ValueError),  # not on a GPU
    ):
        with pytest.raises(err):
            binding.gemm_grouped(*args, **kw)
    with pytest.raises(TypeError):
        binding.gemm_grouped_weights(z(4, 8, **h), z(4, 8), off)
    with pytest.raises(ValueError):
        binding.gemm_grouped_weights(z(4, 8, **h), z(5, 8, **h), off)
    with pytest.raises(ValueError):
        binding.gemm_grouped_weights(z(4, 8, **h), z(4, 8, **h), off, z(2, 8, 8))
    with pytest.raises(ValueError):
        binding.gemm_group_rows(z(2, 2, 2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        binding.gemm_group_rows(z(4), 4, off, off, off)
    with pytest.raises(TypeError):
        binding.gemm_orthogonalize(z(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.gemm_orthogonalize(z(4))
    with pytest.raises(ValueError):
        binding.gemm_orthogonalize(z(4, 4), z(4, 5))
    with pytest.raises(TypeError):
        binding.gemm_orthogonalize(z(4, 4), z(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.gemm_orthogonalize(z(4, 4), z(4, 4))  # not on a GPU


def test_stack_pitches():
    """One row's pitch says nothing, nor the stride of one matrix: the C checks see values they accept."""
    x = torch.zeros(3, 1, 24, dtype=torch.bfloat16)[:, :, :20]
    _, ld, stride = binding._stack("x", x, 3, 1, 20, torch.bfloat16)
    assert stride == 24 and ld == 24
    y = torch.zeros(1, 1, 21, dtype=torch.bfloat16)
    _, ld, _ = binding._stack("y", y, 1, 1, 21, torch.bfloat16)
    assert ld == 24


def _calls():
    """Every wrapper that makes its outputs where it is given none: (call, number of new tensors)."""
    z, h = torch.zeros, dict(dtype=torch.bfloat16)
    u8 = dict(dtype=torch.uint8)
    A, B, C, off = z(4, 32, **h), z(8, 32, **h), z(4, 8), z(4, dtype=torch.int32)
    W, q, s, G = z(3, 8, 32, **h), z(4, 16, **u8), z(1, 4, **u8), z(4, 8, **h)
    b = binding
    return {
        "gemm": (lambda **k: b.gemm(A, B, C, **k), 1),
        "gemm_f16": (lambda **k: b.gemm_f16(A.half(), B.half(), **k), 1),
        "gemm_gather_rows": (lambda **k: b.gemm_gather_rows(A, off, B, **k), 1),
        "gemm_seeded": (lambda **k: b.gemm_seeded(A, B, C, **k), 1),
        "gemm_skinny_noalloc": (lambda **k: b.gemm_skinny_noalloc(A, B, **k), 1),
        "gemm_bf16_e2m1": (lambda **k: b.gemm_bf16_e2m1(A, q, s, **k), 1),
        "gemm_e2m1": (lambda **k: b.gemm_e2m1(q, s, q, s, **k), 1),
        "gemm_gated": (lambda **k: b.gemm_gated(A, B, B, **k), 1),
        "gemm_gated_e2m1": (lambda **k: b.gemm_gated_e2m1(q, s, q, s, q, s, **k), 1),
        "gemm_gated_backward": (lambda **k: b.gemm_gated_backward(G, G, G, A, B, B, **k), 5),
        "gemm_trans": (lambda **k: b.gemm_trans(A, B, **k), 1),
        "gemm_quantize_e2m1": (lambda **k: b.gemm_quantize_e2m1(A, **k), 2),
        "gemm_group_rows": (lambda **k: b.gemm_group_rows(off, 3, **k), 3),
        "gemm_grouped": (lambda **k: b.gemm_grouped(A, W, off, **k), 1),
        "gemm_grouped_weights": (lambda **k: b.gemm_grouped_weights(A, A, off, **k), 1),
        "gemm_orthogonalize": (lambda **k: b.gemm_orthogonalize(A, **k), 1),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_new_outputs_belong_to_the_stream_of_the_call(monkeypatch, name):
    """torch gives a stream's freed memory to that stream again while its kernels may still use it: an
    output that another stream writes has to come from that stream's memory."""
    call, count = _calls()[name]

    class Stream:
        cuda_stream = 0x70

    class Context:
        def __enter__(self):
            where.append(stream)

        def __exit__(self, *_):
            where.pop()

    class Library:
        def __getattr__(self, entry):
            return lambda *args: used.append(args[-1]) or 0

    stream, where, made, used = Stream(), [None], [], []
    monkeypatch.setattr(binding, "load_library", lambda: Library())
    monkeypatch.setattr(binding, "_on_device", lambda *t: None)
    monkeypatch.setattr(binding, "_on_stream", lambda s: Context() if s is stream else pytest.fail("another stream"))
    for made_by in ("empty", "empty_strided"):
        real = getattr(torch, made_by)
        monkeypatch.setattr(torch, made_by, lambda *a, real=real, **k: made.append(where[-1]) or real(*a, **k))
    call(stream=stream)
    assert made == [stream] * count and used == [stream.cuda_stream]


def test_inject_modes(lib):
    assert [lib.gemm_debug_inject(m) for m in (2, 1, 3, -1, 0)] == [0, 0, 1, 1, 0]


@pytest.mark.parametrize("depth", [1, 3])
def test_single_rows_far_apart(depth):
    """The pitch of a matrix of one row is made up: it does not pass the limit of pitches (2^31 - 1) where the
    matrices, or a slice's rows, lie further apart than that."""
    far = (1 << 31) + 8
    x = torch.empty_strided((depth, 1, 20), (far, far, 1), dtype=torch.bfloat16, device="meta")
    _, ld, stride = binding._stack("x", x, depth, 1, 20, torch.bfloat16)
    assert ld == 24 and stride == far
    if depth == 1:
        assert binding._mat("x", x[0], 1, 20, torch.bfloat16)[1] == 24
