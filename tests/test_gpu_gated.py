"""gemm_gated, gemm_gated_e2m1 and gemm_gated_backward against their 64-bit forms (needs a GB300).

Bounds are those of gated_ref.  With quarter-integer inputs and relu, G and U are exact in
float32 whatever the order of the sum and D is one float32 product, so those cases compare
bit for bit on every kernel form.
"""
import numpy as np
import pytest
import torch

import gated_ref as ref
from gated_ref import ACTS, assert_close, wide
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding
from tensor_core_gemm_02_gb300.workloads import OUT_BF16, OUT_F16, OUT_F32

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
FORMS = {"auto": (0, 0), "single64": (1, 64), "single128": (1, 128), "single256": (1, 256),
         "pair": (3, 256), "skinny": (2, 0)}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(seed, M, N, K, dtype, exact=False, scale=0.05):
    r = gen(seed)
    return (wide(M, K, dtype, r, exact=exact), wide(N, K, dtype, r, 1.0 if exact else scale, exact=exact),
            wide(N, K, dtype, r, 1.0 if exact else scale, exact=exact))


def bits(x):
    return x.detach().float().cpu().numpy()


def exact_relu(A, Bg, Bu, dtype):
    """float32 bits of relu(G) * U (G, U exact), rounded to `dtype`."""
    _, g, u, _, _ = ref.gated64(A, Bg, Bu, "relu")
    d = torch.from_numpy(np.maximum(g.numpy().astype(np.float32), np.float32(0)) * u.numpy().astype(np.float32))
    return d.to(dtype).float().numpy(), g, u


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 64), (2, 63, 65), (17, 200, 520), (64, 129, 1000),
                                   (33, 4100, 136)])
def test_exact_few_rows(form, M, N, K):
    binding.gemm_debug_force_tile(*FORMS[form])
    for dtype, out in ((BF16, OUT_F32), (F16, OUT_BF16), (BF16, OUT_F16)):
        A, Bg, Bu = inputs(M + N + K, M, N, K, dtype, exact=True)
        want, _, _ = exact_relu(A, Bg, Bu, ref.out_dtype(out))
        got = binding.gemm_gated(A, Bg, Bu, act="relu", out=out)
        assert np.array_equal(bits(got), want), (form, dtype, out)


@pytest.mark.parametrize("form", [f for f in FORMS if f != "skinny"])
@pytest.mark.parametrize("M,N,K", [(65, 64, 64), (129, 130, 72), (256, 128, 256), (300, 520, 200),
                                   (700, 1001, 328)])
def test_exact_every_tile_form_keeps_both_products(form, M, N, K):
    binding.gemm_debug_force_tile(*FORMS[form])
    for dtype in (BF16, F16):
        A, Bg, Bu = inputs(M * 3 + N + K, M, N, K, dtype, exact=True)
        want, g, u = exact_relu(A, Bg, Bu, torch.float32)
        G = wide(M, N, dtype, gen(1))
        U = wide(M, N, dtype, gen(2))
        got = binding.gemm_gated(A, Bg, Bu, G=G, U=U, act="relu")
        assert np.array_equal(bits(got), want)
        assert np.array_equal(bits(G), g.float().to(dtype).float().numpy())
        assert np.array_equal(bits(U), u.float().to(dtype).float().numpy())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K,dtype,out", [(1, 1000, 4096, BF16, OUT_F32), (16, 2048, 2048, F16, OUT_F16),
                                             (48, 700, 4096, BF16, OUT_BF16), (200, 300, 1000, F16, OUT_F32),
                                             (600, 264, 2056, BF16, OUT_BF16)])
def test_random_within_bound(act, M, N, K, dtype, out):
    A, Bg, Bu = inputs(M + N, M, N, K, dtype, scale=2.0 / K ** 0.5)
    d, g, u, tg, tu = ref.gated64(A, Bg, Bu, act)
    got = binding.gemm_gated(A, Bg, Bu, act=act, out=out)
    assert_close(got, d, ref.gated_bound(act, K, d, g, u, tg, tu, out), f"{act} {M}x{N}x{K}")


@pytest.mark.parametrize("act", ACTS)
def test_large_products(act):
    """G of hundreds either way: exponentials overflow and underflow, results stay finite."""
    A, Bg, Bu = inputs(5, 130, 96, 256, BF16, scale=12.0)
    d, g, u, tg, tu = ref.gated64(A, Bg, Bu, act)
    got = binding.gemm_gated(A, Bg, Bu, act=act)
    assert torch.isfinite(got).all() and g.abs().max() > 300
    assert_close(got, d, ref.gated_bound(act, 256, d, g, u, tg, tu, OUT_F32), act)


@pytest.mark.parametrize("M", [3, 100])
def test_unaligned_output_and_one_kept(M):
    """D, G and U at odd addresses and pitches (plain stores); only one product kept; columns
    past N and rows past M stay as they were."""
    N, K = 77, 96
    A, Bg, Bu = inputs(11, M, N, K, F16, exact=True)
    want, g, u = exact_relu(A, Bg, Bu, F16)
    for keep in ("G", "U", "both", "none"):
        buf = [torch.full((M + 1, N + 5), 9.0, dtype=F16, device="cuda") for _ in range(3)]
        D, G, U = (b[:M, 3:3 + N] for b in buf)
        kw = {"G": {"G": G}, "U": {"U": U}, "both": {"G": G, "U": U}, "none": {}}[keep]
        binding.gemm_gated(A, Bg, Bu, D, act="relu", out=OUT_F16, **kw)
        assert np.array_equal(bits(D), want)
        for t, b, r, name in ((D, buf[0], None, "D"), (G, buf[1], g, "G"), (U, buf[2], u, "U")):
            if r is not None and name in kw:
                assert np.array_equal(bits(t), r.float().to(F16).float().numpy())
            b[:M, 3:3 + N] = 9.0
            assert (b == 9.0).all(), f"{name} written outside"


def test_k_zero_and_empty():
    e = torch.empty((5, 0), dtype=BF16, device="cuda")
    w = torch.empty((9, 0), dtype=BF16, device="cuda")
    for act in ACTS:
        G = torch.ones((5, 9), dtype=BF16, device="cuda")
        D = binding.gemm_gated(e, w, w, torch.ones((5, 9), device="cuda"), G=G, act=act)
        assert (D == 0).all() and (G == 0).all()
    assert binding.gemm_gated(torch.empty((0, 8), dtype=BF16, device="cuda"),
                              torch.ones((4, 8), dtype=BF16, device="cuda"),
                              torch.ones((4, 8), dtype=BF16, device="cuda")).shape == (0, 4)


@pytest.mark.parametrize("M,form", [(4, "skinny"), (4, "single128"), (300, "pair")])
def test_nan_and_infinity_stay_in_their_rows_and_columns(M, form):
    binding.gemm_debug_force_tile(*FORMS[form])
    N, K = 200, 264
    A, Bg, Bu = inputs(3, M, N, K, BF16, exact=True)
    A[1, 7] = float("nan")
    Bu[5, 9] = float("inf")
    D = binding.gemm_gated(A, Bg, Bu, act="relu")
    A[1, 7] = 0
    Bu[5, 9] = 0
    clean = binding.gemm_gated(A, Bg, Bu, act="relu")
    assert torch.isnan(D[1]).all()
    keep = torch.ones((M, N), dtype=torch.bool, device="cuda")
    keep[1], keep[:, 5] = False, False
    assert torch.equal(D[keep], clean[keep])


@pytest.mark.parametrize("M", [8, 500])
def test_other_stream_graph_and_repeats(M):
    """The caller's stream is used; a captured graph replays on new inputs; repeated calls give
    the same bits."""
    A, Bg, Bu = inputs(21, M, 1024, 2048, BF16)
    first = binding.gemm_gated(A, Bg, Bu, out=OUT_BF16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    D = torch.empty_like(first)
    s.wait_stream(torch.cuda.current_stream())
    binding.gemm_gated(A, Bg, Bu, D, out=OUT_BF16, stream=s)
    s.synchronize()
    assert torch.equal(D, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.gemm_gated(A, Bg, Bu, D, out=OUT_BF16)
    A.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D, binding.gemm_gated(A, Bg, Bu, out=OUT_BF16)) and not torch.equal(D, first)


@pytest.mark.parametrize("form", ["single128", "pair", "skinny", "fp4_skinny", "fp4_128", "fp4_256"])
def test_timeout_reports_and_recovers(form):
    M = 16 if "skinny" in form else 300
    A, Bg, Bu = inputs(2, M, 512, 1024, BF16, exact=True)
    if form.startswith("fp4"):
        if M > 64:
            binding.gemm_debug_force_tile(11, int(form[4:]))
        q = [x for t in (A, Bg, Bu) for x in binding.gemm_quantize_e2m1(t)]
        call = lambda: binding.gemm_gated_e2m1(*q, act="relu")  # noqa: E731
    else:
        binding.gemm_debug_force_tile(*FORMS[form])
        call = lambda: binding.gemm_gated(A, Bg, Bu, act="relu")  # noqa: E731
    good = call()
    assert device_status() == binding.GEMM_OK
    binding.gemm_set_wait_timeout(50_000_000)
    binding.gemm_debug_inject(1)
    try:
        call()
        assert device_status() == binding.GEMM_ERR_TIMEOUT
    finally:
        binding.gemm_debug_inject(0)
        binding.gemm_set_wait_timeout(0)
    assert torch.equal(call(), good)


# ---------------------------------------------------------------- FP4

FP4_FORMS = {"auto": (0, 0), "tile256": (11, 256), "tile128": (11, 128)}


def fp4_inputs(seed, M, N, K):
    r = np.random.default_rng(seed)
    mats = []
    for rows in (M, N, N):
        codes = r.choice(np.array([0, 1, 2, 3, 4, 8, 9, 10, 11, 12]), (rows, K))
        scales = r.integers(126, 129, (K // 32, rows)).astype(np.uint8)
        mag = np.where(codes & 8, -1, 1) * ref.LEVELS[codes & 7]
        values = mag * np.repeat(np.ldexp(1.0, scales.astype(int) - 127).T, 32, axis=1)
        mats.append((torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda(),
                     torch.from_numpy(values)))
    return mats


@pytest.mark.parametrize("form", FP4_FORMS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 64, 256), (16, 200, 4096), (40, 65, 544), (64, 1500, 2048),
                                   (65, 64, 64), (130, 257, 288), (300, 520, 1024), (700, 130, 96)])
def test_fp4_exact(form, M, N, K):
    binding.gemm_debug_force_tile(*FP4_FORMS[form])
    (aq, as_, a), (gq, gs, bg), (uq, us, bu) = fp4_inputs(M + N + K, M, N, K)
    for out in (OUT_F32, OUT_BF16, OUT_F16):
        want, _, _ = exact_relu(a, bg, bu, ref.out_dtype(out))
        got = binding.gemm_gated_e2m1(aq, as_, gq, gs, uq, us, act="relu", out=out)
        assert np.array_equal(bits(got), want), (form, out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 190])
def test_fp4_quantised_activations_within_bound(act, M):
    """The serving path: activations quantised, then the gated block on their codes."""
    N, K = 300, 2048
    r = gen(M)
    X, Wg, Wu = wide(M, K, BF16, r), wide(N, K, BF16, r, 0.04), wide(N, K, BF16, r, 0.04)
    vals, q = [], []
    for t in (X, Wg, Wu):
        y = torch.empty_like(t)
        q += list(binding.gemm_quantize_e2m1(t, Y=y))
        vals.append(y)
    d, g, u, tg, tu = ref.gated64(*vals, act)
    got = binding.gemm_gated_e2m1(*q, act=act, out=OUT_BF16)
    assert_close(got, d, ref.gated_bound(act, K, d, g, u, tg, tu, OUT_BF16), act)


@pytest.mark.parametrize("M", [7, 200])
def test_fp4_unaligned_scales_and_nan_scale(M):
    N, K = 90, 256
    (aq, as_, a), (gq, gs, bg), (uq, us, bu) = fp4_inputs(4, M, N, K)
    odd = []
    for s in (as_, gs, us):
        b = torch.zeros((s.shape[0], s.shape[1] + 7), dtype=torch.uint8, device="cuda")
        b[:, 3:3 + s.shape[1]] = s
        odd.append(b[:, 3:3 + s.shape[1]])
    want, _, _ = exact_relu(a, bg, bu, torch.float32)
    got = binding.gemm_gated_e2m1(aq, odd[0], gq, odd[1], uq, odd[2], act="relu")
    assert np.array_equal(bits(got), want)
    odd[0][3, 2] = 255  # block 3 of row 2 of A
    got = bits(binding.gemm_gated_e2m1(aq, odd[0], gq, odd[1], uq, odd[2], act="relu"))
    assert np.isnan(got[2]).all()
    keep = np.arange(M) != 2
    assert np.array_equal(got[keep], want[keep])


# ---------------------------------------------------------------- gradients

def backward_inputs(seed, M, N, K, dtype, scale=0.05):
    r = gen(seed)
    return dict(dD=wide(M, N, dtype, r), G=wide(M, N, dtype, r, 1.5), U=wide(M, N, dtype, r),
                A=wide(M, K, dtype, r), Bg=wide(N, K, dtype, r, scale), Bu=wide(N, K, dtype, r, scale))


def check_products(x, dA, dBg, dBu, dG, dU, out, what):
    """The three products against 64-bit ones of the dG and dU they were computed from."""
    dg, du = dG.cpu().double(), dU.cpu().double()
    a, bg, bu = (x[k].cpu().double() for k in ("A", "Bg", "Bu"))
    M, N = dg.shape
    for got, want, t, terms in (
            (dA, dg @ bg + du @ bu, dg.abs() @ bg.abs() + du.abs() @ bu.abs(), 2 * N),
            (dBg, dg.T @ a, dg.abs().T @ a.abs(), M), (dBu, du.T @ a, du.abs().T @ a.abs(), M)):
        e = ref.sum_bound(terms) * t
        assert_close(got, want, e + ref.rounding(want.abs() + e, out), what)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K,dtype,out", [(1, 64, 64, BF16, OUT_F32), (50, 130, 72, F16, OUT_F16),
                                             (129, 520, 200, BF16, OUT_BF16), (700, 267, 1001, F16, OUT_F32)])
def test_gradients_against_the_formula(act, M, N, K, dtype, out):
    x = backward_inputs(M + N, M, N, K, dtype)
    dA, dBg, dBu, dG, dU = binding.gemm_gated_backward(**x, act=act, out=out)
    d, g, u = (x[k].cpu().double() for k in ("dD", "G", "U"))
    kind = OUT_BF16 if dtype == BF16 else OUT_F16
    y = ref.argument(act, g, slope=True)
    fp32 = (32 + 16 * y) * 2.0 ** -23
    # the slope's terms cancel near its zeros: its error is relative to their sizes, 1 + |g|
    eg = (d * u).abs() * (1 + g.abs()) * fp32
    eu = d.abs() * (ref.act64(act, g).abs() * fp32 + 4 * 2.0 ** -23 * g.abs())
    want = d * u * ref.slope64(act, g)
    assert_close(dG, want, eg + ref.rounding(want.abs() + eg, kind), f"dG {act}")
    want = d * ref.act64(act, g)
    assert_close(dU, want, eu + ref.rounding(want.abs() + eu, kind), f"dU {act}")
    check_products(x, dA, dBg, dBu, dG, dU, out, act)


@pytest.mark.parametrize("M,N,K,dtype", [(1, 2048, 1032, BF16), (16, 1367, 1000, F16), (33, 3000, 520, BF16),
                                         (64, 4096, 264, F16)])
def test_gradients_of_few_tokens(M, N, K, dtype):
    """dA's long sum on the swap-AB kernel, both sources in one list of K blocks."""
    x = backward_inputs(M + K, M, N, K, dtype)
    for form in ((0, 0), (2, 0)):
        binding.gemm_debug_force_tile(*form)
        check_products(x, *binding.gemm_gated_backward(**x, out=OUT_F32), OUT_F32, str(form))


@pytest.mark.parametrize("M,N,K,dtype", [(200, 3000, 136, BF16), (4100, 130, 72, F16), (2050, 300, 520, BF16)])
def test_gradients_with_sums_in_parts(M, N, K, dtype):
    """Long sums over few tiles (dA's over 2 N, the weight gradients' over M): both products in
    parts, each in a buffer of its own, twice in a row."""
    x = backward_inputs(M + N, M, N, K, dtype)
    first = binding.gemm_gated_backward(**x, out=OUT_F32)
    check_products(x, *first, OUT_F32, "in parts")
    for a, b in zip(first, binding.gemm_gated_backward(**x, out=OUT_F32)):
        assert torch.equal(a, b)


def test_fp4_long_output_under_repeats():
    """A large float32 result keeps HBM busy with stores while loads are late: forty launches, each
    equal to the first and without a wait that ran out."""
    r = gen(12)
    q = [x for n, s in ((2048, 1.0), (8192, 0.05), (8192, 0.05))
         for x in binding.gemm_quantize_e2m1(torch.randn((n, 1024), generator=r).mul(s).cuda())]
    first = binding.gemm_gated_e2m1(*q)
    for _ in range(40):
        D = torch.full_like(first, float("nan"))
        assert torch.equal(binding.gemm_gated_e2m1(*q, D), first)
    assert device_status() == binding.GEMM_OK


@pytest.mark.parametrize("form", ["single64", "single128", "single256", "pair", "pair512"])
def test_gradients_every_form(form):
    binding.gemm_debug_force_tile(*{"pair512": (4, 512)}.get(form, FORMS.get(form)))
    x = backward_inputs(8, 300, 520, 328, BF16)
    check_products(x, *binding.gemm_gated_backward(**x), OUT_F32, form)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Central differences of the loss sum(dD * D) in 64 bits along a random direction of each
    input.  G and U are small dyadic numbers, kept exactly, so what separates the two is the
    rounding of dG and dU to bf16 (2^-9 of each), float32, and the step's own error."""
    M, N, K, h = 24, 40, 16, 2.0 ** -12
    r = gen(17)
    A = (torch.randint(-2, 3, (M, K), generator=r).double() / 2).to(BF16)
    Bg, Bu = ((torch.randint(-2, 3, (N, K), generator=r).double() / 4).to(BF16) for _ in range(2))
    dD = (torch.randint(-8, 9, (M, N), generator=r).double() / 8).to(BF16)
    G, U = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty((M, N), dtype=BF16, device="cuda")
    binding.gemm_gated(A.cuda(), Bg.cuda(), Bu.cuda(), G=G, U=U, act=act)
    if act == "relu":
        dD = torch.where(G.cpu() == 0, torch.zeros_like(dD), dD)  # keep clear of relu's corner
    a, bg, bu, dd = A.double(), Bg.double(), Bu.double(), dD.double()
    assert torch.equal(G.cpu().double(), a @ bg.T) and torch.equal(U.cpu().double(), a @ bu.T)
    dA, dBg, dBu, dG, dU = binding.gemm_gated_backward(dD.cuda(), G, U, A.cuda(), Bg.cuda(), Bu.cuda(), act=act)
    dg, du = dG.cpu().double().abs(), dU.cpu().double().abs()
    loss = lambda a, bg, bu: (dd * ref.act64(act, a @ bg.T) * (a @ bu.T)).sum().item()  # noqa: E731
    for grad, i, t in ((dA, 0, dg @ bg.abs() + du @ bu.abs()), (dBg, 1, dg.T @ a.abs()), (dBu, 2, du.T @ a.abs())):
        v = torch.randn(grad.shape, generator=r, dtype=torch.float64)
        at = [a, bg, bu]
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.cpu().double() * v).sum().item()
        # the differences' own error, h^2 / 6 times the third derivative of act(g) u: |act''| and
        # |act'''| stay below 2
        p = {0: lambda: v @ bg.T, 1: lambda: a @ v.T}.get(i, lambda: torch.zeros(M, N).double())().abs()
        q = {0: lambda: v @ bu.T, 2: lambda: a @ v.T}.get(i, lambda: torch.zeros(M, N).double())().abs()
        step = h * h / 6 * (dd.abs() * (2 * p ** 3 * (a @ bu.T).abs() + 6 * p * p * q)).sum().item()
        step = step + 2.0 ** -40 / h * dd.abs().sum().item()  # the losses' roundings
        bound = (2.0 ** -9 + 2.0 ** -15) * (t * v.abs()).sum().item() + step
        assert abs(got - diff) <= bound, (act, i, got, diff, bound)


def test_gradients_in_place_partial_and_empty():
    x = backward_inputs(31, 70, 96, 64, BF16)
    full = binding.gemm_gated_backward(**x)
    G, U = x["G"].clone(), x["U"].clone()
    y = dict(x, G=G, U=U)
    inplace = binding.gemm_gated_backward(**y, dG=G, dU=U)
    for a, b in zip(full, inplace):
        assert torch.equal(a, b)
    dA, dBg, dBu, _, _ = binding.gemm_gated_backward(**dict(x, A=None), need_weights=False)
    assert dBg is None and dBu is None and torch.equal(dA, full[0])
    dA, dBg, dBu, _, _ = binding.gemm_gated_backward(**dict(x, Bg=None, Bu=None), need_input=False)
    assert dA is None and torch.equal(dBg, full[1]) and torch.equal(dBu, full[2])
    e = backward_inputs(1, 0, 96, 64, BF16)
    dA, dBg, dBu, _, _ = binding.gemm_gated_backward(**e, dBg=torch.ones((96, 64), device="cuda"),
                                                     dBu=torch.ones((96, 64), device="cuda"))
    assert dA.shape == (0, 64) and (dBg == 0).all() and (dBu == 0).all()
    e = backward_inputs(1, 70, 0, 64, BF16)
    dA, dBg, _, _, _ = binding.gemm_gated_backward(**e, dA=torch.ones((70, 64), device="cuda"))
    assert (dA == 0).all() and dBg.shape == (0, 64)


def test_gradients_unaligned_inputs_and_nan_rows():
    """dD, G and U at odd addresses (element loads); a NaN of dD reaches its row of dA and, of the
    weight gradients, its own row only."""
    M, N, K = 33, 45, 64
    x = backward_inputs(9, M, N, K, F16)
    want = binding.gemm_gated_backward(**x)
    odd = {}
    for k in ("dD", "G", "U"):
        b = torch.zeros((M, N + 6), dtype=F16, device="cuda")
        b[:, 3:3 + N] = x[k]
        odd[k] = b[:, 3:3 + N]
    for a, b in zip(want, binding.gemm_gated_backward(**dict(x, **odd))):
        assert torch.equal(a, b)
    odd["dD"][4, 6] = float("nan")
    dA, dBg, dBu, dG, dU = binding.gemm_gated_backward(**dict(x, **odd))
    rows, cols = torch.arange(M) != 4, torch.arange(N) != 6
    assert torch.isnan(dA[4]).all() and torch.equal(dA[rows.cuda()], want[0][rows.cuda()])
    for got, ok in ((dBg, want[1]), (dBu, want[2])):
        assert torch.isnan(got[6]).all() and torch.equal(got[cols.cuda()], ok[cols.cuda()])


def odd_rows(M, N, out):
    """An M x N output whose rows are not 16 bytes apart, in a buffer of NaNs, and that buffer."""
    dtype = {OUT_F32: torch.float32, OUT_BF16: BF16, OUT_F16: F16}[out]
    b = torch.full((M + 1, N + 9 - N % 8), float("nan"), dtype=dtype, device="cuda")
    return b[:M, 1:1 + N], b


@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16, OUT_F16])
@pytest.mark.parametrize("M,N,K", [(32, 33, 64), (191, 300, 128), (300, 129, 320)])
def test_output_rows_not_16_bytes_apart(out, M, N, K):
    """D (and kept G) written without TMA, on every tile form: the same bits as an aligned D,
    nothing beside it."""
    A, Bg, Bu = inputs(M, M, N, K, F16)
    fp4 = [t for m in (A, Bg, Bu) for t in binding.gemm_quantize_e2m1(m)]
    calls = [(FORMS[f], lambda D, **kw: binding.gemm_gated(A, Bg, Bu, D, act="gelu", out=out, **kw))
             for f in ("single64", "single128", "single256", "pair")]
    calls += [((11, bn), lambda D: binding.gemm_gated_e2m1(*fp4, D, act="gelu", out=out)) for bn in (128, 256)]
    for form, call in calls:
        binding.gemm_debug_force_tile(*form)
        want = call(None) if N % 8 == 0 else call(torch.empty((M, N + 8 - N % 8), dtype=odd_rows(1, N, out)[0].dtype,
                                                              device="cuda")[:, :N])
        for keep in ((False, True) if form[0] != 11 else (False,)):
            D, buf = odd_rows(M, N, out)
            G, gbuf = odd_rows(M, N, OUT_F16)
            call(D, G=G) if keep else call(D)
            assert np.array_equal(bits(D), bits(want)), (form, keep)
            assert int(torch.isnan(buf).sum()) == buf.numel() - M * N
            if keep:
                K_aligned = torch.empty((M, N + 8 - N % 8), dtype=F16, device="cuda")[:, :N]
                call(D, G=K_aligned)
                assert np.array_equal(bits(G), bits(K_aligned)), form
                assert int(torch.isnan(gbuf).sum()) == gbuf.numel() - M * N


@pytest.mark.parametrize("bn", [128, 256])
def test_fp4_more_block_rows_than_a_group(bn):
    """M past 64 block rows (a full group of the tile order and a part of one), bit for bit."""
    M, N, K = 8450, 130, 96
    (aq, as_, a), (gq, gs, bg), (uq, us, bu) = fp4_inputs(5, M, N, K)
    want, _, _ = exact_relu(a, bg, bu, BF16)
    binding.gemm_debug_force_tile(11, bn)
    assert np.array_equal(bits(binding.gemm_gated_e2m1(aq, as_, gq, gs, uq, us, act="relu", out=OUT_BF16)), want)


@pytest.mark.parametrize("M,N,K,dtype", [(1000, 1367, 1000, F16), (512, 2000, 800, BF16), (1500, 700, 700, BF16)])
def test_gradients_planned_side_by_side(M, N, K, dtype):
    """Both products of a size where the weights' one keeps to the SMs that the input's leaves."""
    x = backward_inputs(M, M, N, K, dtype)
    check_products(x, *binding.gemm_gated_backward(**x), OUT_F32, (M, N, K))


MIXES = {"GU|d": ("GU", "D"), "G|d": ("G", "D"), "U|d": ("U", "D"), "D|gu": ("D", "GU"), "D|g": ("D", "G"),
         "D|u": ("D", "U")}


@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16, OUT_F16])
@pytest.mark.parametrize("form", ["single64", "single128", "single256", "pair"])
def test_outputs_of_mixed_alignment(form, out):
    """D, G and U of one call, some with rows 16 bytes apart (stored by TMA) and some not (copied), over
    several chunks and tiles per CTA: every one bit for bit, nothing beside it."""
    M, N, K = 1300, 4001, 64
    A, Bg, Bu = inputs(7, M, N, K, BF16, exact=True)
    d, g, u = exact_relu(A, Bg, Bu, ref.out_dtype(out))
    want = {"D": d, "G": g.bfloat16().float().numpy(), "U": u.bfloat16().float().numpy()}
    binding.gemm_debug_force_tile(*FORMS[form])
    for name, (aligned, odd) in MIXES.items():
        for _ in range(3):
            x, bufs = {}, {}
            for k in aligned:
                dtype = ref.out_dtype(out) if k == "D" else BF16
                bufs[k] = torch.full((M, (N + 7) // 8 * 8), float("nan"), dtype=dtype, device="cuda")
                x[k] = bufs[k][:, :N]
            for k in odd:
                x[k], bufs[k] = odd_rows(M, N, out if k == "D" else OUT_BF16)
            binding.gemm_gated(A, Bg, Bu, act="relu", out=out, **x)
            for k in x:
                assert np.array_equal(bits(x[k]), want[k]), (name, k)
                assert int(torch.isnan(bufs[k]).sum()) == bufs[k].numel() - M * N, (name, k)
