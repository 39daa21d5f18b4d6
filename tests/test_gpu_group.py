"""Grouped rows, grouped products and the gradients of the groups' weights on the GPU (needs a
GB300): quarter-integers compare bit for bit with 64-bit sums (every partial sum is exact in
float32), normal inputs within gated_ref's sum bound, whole numbers exactly."""
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
FORMS = {"auto": (0, 0), "few": (2, 0), "single64": (1, 64), "single128": (1, 128), "single256": (1, 256), "pair256": (3, 256)}
KINDS = ((BF16, OUT_F32), (F16, OUT_BF16), (BF16, OUT_F16))
# rows of each group, and rows outside every group in front and behind
GROUPS = {
    "one": ([37], 0, 0),
    "even": ([128, 128, 128], 0, 0),
    "ragged": ([1, 0, 257, 64, 0, 0, 300, 5], 3, 20),
    "tails": ([15, 16, 17, 63, 65, 127, 129, 31], 0, 1),
    "none": ([0, 0, 0], 0, 9),
    "many": ([(7 * i) % 23 for i in range(130)], 2, 2),
}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK


def sum_bound(K, out):
    """As gated_ref's; float32 results are added up in registers every 512 of K, each time one rounding."""
    return ref.sum_bound(K) if out != OUT_F32 else ref.sum_bound(min(K, 512)) + K / 512 * 2.0 ** -24


def offsets_of(counts, front):
    return torch.tensor(np.cumsum([front] + list(counts)), dtype=torch.int32, device="cuda")


def bounds(counts, front):
    b = np.cumsum([front] + list(counts)).tolist()
    return list(zip(b[:-1], b[1:]))


def stack(e, rows, cols, dtype, gen, exact, scale=1.0):
    """A stack of slices of wider buffers, whose padding is NaN, with rows of padding between matrices."""
    x = wide(e * (rows + 1), cols, dtype, gen, scale=scale, exact=exact)
    return torch.as_strided(x, (e, rows, cols), ((rows + 1) * x.stride(0), x.stride(0), 1))


def grouped64(A, B, counts, front, trans_b):
    """(D, sum |a||b|) of the rows of the groups, NaN elsewhere, in 64 bits."""
    a, b = A.cpu().double(), B.cpu().double()
    N = b.shape[2] if trans_b else b.shape[1]
    d, t = (torch.full((a.shape[0], N), float("nan"), dtype=torch.float64) for _ in range(2))
    for g, (lo, hi) in enumerate(bounds(counts, front)):
        w = b[g] if trans_b else b[g].T
        d[lo:hi], t[lo:hi] = a[lo:hi] @ w, a[lo:hi].abs() @ w.abs()
    return d, t


def new_out(M, N, out, pad=8, fill=7.0):
    ld = (N + 7) // 8 * 8 + pad
    return torch.full((M, ld), fill, dtype=ref.out_dtype(out), device="cuda")


def check_grouped(counts, front, behind, N, K, trans_b, dtype, out, exact, seed=0, idx=False, pad=8):
    gen = torch.Generator().manual_seed(seed + N + K)
    M = front + sum(counts) + behind
    B = stack(len(counts), K if trans_b else N, N if trans_b else K, dtype, gen, exact)
    if idx:
        table = wide(max(1, M // 3), K, dtype, gen, exact=exact)
        rows = torch.randint(0, table.shape[0], (M,), generator=gen).int()
        A, given = table[rows.long().cuda()], dict(idx=rows.cuda())
    else:
        table, given = wide(M, K, dtype, gen, exact=exact), {}
        A = table
    buf = new_out(M, N, out, pad)
    D = buf[:, :N]
    alpha = 0.5
    got = binding.gemm_grouped(table, B, offsets_of(counts, front), D, trans_b=trans_b, alpha=alpha, out=out, **given)
    assert got is D
    s, t = grouped64(A, B, counts, front, trans_b)
    inside = torch.zeros(M, dtype=torch.bool)
    inside[front:front + sum(counts)] = True
    what = (counts, N, K, trans_b, dtype, out, idx, pad)
    host = buf.cpu().float()
    assert (host[~inside] == 7).all() and (host[:, N:] == 7).all(), what  # nothing else written
    want = alpha * s[inside]
    if exact:
        assert torch.equal(D.cpu()[inside], want.float().to(ref.out_dtype(out))), what
    else:
        b = alpha * sum_bound(K, out) * t[inside] + 2.0 ** -23 * want.abs()
        assert_close(D.cpu()[inside], want, b + ref.rounding(want.abs() + b, out), what)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("groups", GROUPS)
def test_grouped_exact(form, trans_b, groups):
    binding.gemm_debug_force_tile(*FORMS[form])
    counts, front, behind = GROUPS[groups]
    for i, (N, K) in enumerate(((1, 1), (70, 64), (264, 63), (520, 200))):
        dtype, out = KINDS[i % 3]
        check_grouped(counts, front, behind, N, K, trans_b, dtype, out, True, idx=i % 2 == 1 and front + behind + sum(counts) > 0)


@pytest.mark.parametrize("form", FORMS)
def test_grouped_outputs_of_any_pitch(form):
    """Rows of D that are not whole 16 bytes apart, and odd numbers of columns."""
    binding.gemm_debug_force_tile(*FORMS[form])
    counts, front, behind = GROUPS["ragged"]
    for N in (1, 31, 129, 260):
        for dtype, out in KINDS:
            for pad in (0, 1, 3):
                check_grouped(counts, front, behind, N, 72, False, dtype, out, True, pad=pad)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("N", [1, 2, 3, 31, 33, 34, 35, 65, 66, 67, 98, 130, 257, 258])
def test_row_ends_between_words(form, N):
    """Rows of D of an odd pitch end at any place of a piece of 32 or 64 columns; the column behind
    keeps what it holds."""
    binding.gemm_debug_force_tile(*FORMS[form])
    for out in (OUT_F32, OUT_BF16, OUT_F16):
        for exact in (True, False):
            check_grouped([35, 0, 6], 0, 2, N, 24, False, F16, out, exact, pad=1)
            check_weights([35, 0, 6], 0, 2, 24, N, F16, out, exact, pad=1)


@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("counts,N,K", [([700, 3, 0, 900], 777, 1000), ([2, 1, 0, 1] * 8, 1030, 2056),
                                        ([40, 0, 90, 20], 4096, 4100), ([16] * 20, 264, 328), ([64, 1, 33], 130, 8200)])
def test_grouped_normal(trans_b, counts, N, K):
    for dtype, out in ((BF16, OUT_BF16), (F16, OUT_F32)):
        check_grouped(counts, 0, 5, N, K, trans_b, dtype, out, False)
        check_grouped(counts, 0, 0, N, K, trans_b, dtype, out, False, idx=True)


@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 5, 1], [12, 16], [40, 60, 2], [1]])
def test_few_rows_and_long_sums(trans_b, counts):
    """Fewer tiles than half of the SMs: two CTAs share each tile's sum."""
    for i, K in enumerate((4096, 4104, 8200)):
        dtype, out = KINDS[i]
        check_grouped(counts, 0, 2, 200, K, trans_b, dtype, out, True, idx=i == 1)


@pytest.mark.parametrize("form", ["auto", "few"])
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 5, 1], 200, 14336), ([3, 0, 5, 1], 200, 114696), ([12, 16], 130, 65544),
                                        ([40, 30], 130, 65544), ([1] * 80, 8, 57352), ([40] * 80, 8, 28680)])
def test_float32_sums_of_one_sign(form, trans_b, counts, N, K):
    """Positive operands: nothing cancels, and what each step of a long sum drops adds up.  (The last two on
    one CTA a tile, the others on two.)"""
    binding.gemm_debug_force_tile(*FORMS[form])
    gen = torch.Generator().manual_seed(K)
    M = sum(counts)
    A, B = wide(M, K, F16, gen).abs_(), stack(len(counts), K if trans_b else N, N if trans_b else K, F16, gen, False).abs_()
    s, t = grouped64(A, B, counts, 0, trans_b)
    assert torch.equal(s, t)
    D = binding.gemm_grouped(A, B, offsets_of(counts, 0), trans_b=trans_b, alpha=0.5)
    want = 0.5 * s
    b = 0.5 * sum_bound(K, OUT_F32) * t + 2.0 ** -23 * want
    assert_close(D, want, b + ref.rounding(want + b, OUT_F32), (counts, N, K))


def test_grouped_largest_number_of_groups():
    gen = torch.Generator().manual_seed(3)
    counts = torch.randint(0, 4, (1024,), generator=gen).tolist()
    check_grouped(counts, 0, 0, 40, 72, False, BF16, OUT_F32, True)
    check_grouped([0] * 1023 + [200], 0, 0, 40, 72, True, BF16, OUT_F32, True)
    check_grouped([5] + [0] * 1023, 1, 1, 40, 72, False, F16, OUT_F32, True)


@pytest.mark.parametrize("form", FORMS)
def test_rows_of_other_groups_do_not_matter(form):
    """NaN and infinities in one group's rows, and outside every group, stay there."""
    binding.gemm_debug_force_tile(*FORMS[form])
    gen = torch.Generator().manual_seed(5)
    counts, front, behind = [21, 90, 40, 0, 150], 6, 30
    M, N, K = front + sum(counts) + behind, 136, 200
    A, dD = wide(M, K, F16, gen, exact=True), wide(M, N, F16, gen, exact=True)
    B, off = stack(5, N, K, F16, gen, True), offsets_of(counts, front)
    want = binding.gemm_grouped(A, B, off)
    grads = binding.gemm_grouped_weights(dD, A, off)
    bad = torch.zeros(M, dtype=torch.bool)
    bad[:front] = bad[front + 21:front + 111] = bad[front + sum(counts):] = True
    for x in (A, dD):
        x[bad.cuda()] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=F16).repeat(
            x.shape[1] // 3 + 1)[:x.shape[1]]
    got = binding.gemm_grouped(A, B, off)
    good = ~bad
    assert torch.equal(got.cpu()[good], want.cpu()[good])
    assert torch.isnan(got.cpu()[front + 21:front + 111]).any()
    got = binding.gemm_grouped_weights(dD, A, off)
    for g in (0, 2, 3, 4):
        assert torch.equal(got[g], grads[g]), g
    assert not torch.isfinite(got[1]).any()  # (infinities of one sign add up to infinity)


def test_no_columns_to_sum():
    off = offsets_of([3, 0, 4], 1)
    D = torch.full((10, 24), 7.0, device="cuda")
    binding.gemm_grouped(torch.zeros(10, 0, dtype=BF16, device="cuda"), torch.zeros(3, 24, 0, dtype=BF16, device="cuda"),
                         off, D)
    assert (D[1:8] == 0).all() and (D[0] == 7).all() and (D[8:] == 7).all()


@pytest.mark.parametrize("offsets", [[0, 5, 4, 8], [-1, 2, 4, 8], [0, 2, 4, 11], [5, 4, 3, 2]])
def test_bad_offsets_are_reported(offsets):
    """Nothing is written, the device status says why, and the next call works."""
    gen = torch.Generator().manual_seed(1)
    A, B = wide(10, 40, BF16, gen, exact=True), stack(3, 24, 40, BF16, gen, True)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    D = torch.full((10, 24), 7.0, device="cuda")
    binding.gemm_grouped(A, B, off, D)
    assert device_status() == binding.GEMM_ERR_INDEX
    assert (D == 7).all()
    dB = torch.full((3, 24, 40), 7.0, device="cuda")
    binding.gemm_grouped_weights(wide(10, 24, BF16, gen), A, off, dB)
    assert device_status() == binding.GEMM_ERR_INDEX
    assert (dB == 0).all()
    check_grouped([3, 4, 3], 0, 0, 24, 40, False, BF16, OUT_F32, True)


@pytest.mark.parametrize("form", FORMS)
def test_bad_row_indices_make_zero_rows(form):
    binding.gemm_debug_force_tile(*FORMS[form])
    gen = torch.Generator().manual_seed(2)
    table, B = wide(12, 72, F16, gen, exact=True), stack(2, 40, 72, F16, gen, True)
    idx = torch.randint(0, 12, (50,), generator=gen).int()
    off = offsets_of([20, 25], 2)
    want = binding.gemm_grouped(table, B, off, idx=idx.cuda())
    idx[5], idx[30] = 12, -1
    idx[0] = idx[49] = 1 << 30  # (of no group: not read)
    got = binding.gemm_grouped(table, B, off, idx=idx.cuda())
    assert device_status() == binding.GEMM_ERR_INDEX
    want[5] = want[30] = 0
    assert torch.equal(got, want)
    idx[5] = idx[30] = 0
    binding.gemm_grouped(table, B, off, idx=idx.cuda())
    assert device_status() == binding.GEMM_OK


# ---------------------------------------------------------------- the gradients of the weights

# enough tiles that the rows are laid out in order first
GATHERED = [([1500, 0, 700, 801], 5, 30, 2056, 519), ([3] * 100, 0, 7, 4000, 264), ([40] * 30, 2, 0, 3000, 1000), ([4000], 0, 0, 1030, 64)]


@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("counts,front,behind,N,K", GATHERED)
def test_gathered_rows_of_large_calls(trans_b, counts, front, behind, N, K):
    for dtype, out in KINDS:
        check_grouped(counts, front, behind, N, K, trans_b, dtype, out, True, idx=True)
        check_grouped(counts, front, behind, N, K, trans_b, dtype, out, False, idx=True)


def test_more_gathered_rows_than_are_laid_out():
    """Rows of which the workspace would pass 8 GiB are gathered by the product itself."""
    gen = torch.Generator().manual_seed(8)
    M, N, K = (1 << 21) + 128, 8, 2048
    table, B = wide(50, K, F16, gen, exact=True), stack(2, N, K, F16, gen, True)
    idx = torch.randint(0, 50, (M,), generator=gen).int()
    off = torch.tensor([0, 1 << 20, M], dtype=torch.int32, device="cuda")
    D = binding.gemm_grouped(table, B, off, idx=idx.cuda())
    every = torch.stack([table.double() @ b.double().T for b in B])  # (group, row of the table, N)
    g = (torch.arange(M) >= 1 << 20).long()
    assert torch.equal(D, every[g.cuda(), idx.long().cuda()].float())


@pytest.mark.parametrize("counts,front,behind,N,K", GATHERED)
def test_bad_row_indices_of_large_calls(counts, front, behind, N, K):
    """Their rows are zero whatever B holds, and the error is recorded; indices of rows outside every
    group are not read."""
    gen = torch.Generator().manual_seed(5)
    M = front + sum(counts) + behind
    table, B = wide(50, K, F16, gen, exact=True), stack(len(counts), N, K, F16, gen, True)
    idx = torch.randint(0, 50, (M,), generator=gen).int()
    idx[:front] = -5
    idx[M - behind:] = 1 << 30
    idx = idx.cuda()
    off = offsets_of(counts, front)
    D = new_out(M, N, OUT_F32)[:, :N]
    want = binding.gemm_grouped(table, B, off, D, idx=idx).clone()
    assert device_status() == binding.GEMM_OK
    bad = [front, front + 2, front + sum(counts) - 1]
    for i, v in zip(bad, (-1, 50, (1 << 31) - 1)):
        idx[i] = v
        want[i] = 0
    B[:, 0, 0] = float("inf")
    keep = torch.ones(N, dtype=torch.bool)
    keep[0] = False
    binding.gemm_grouped(table, B, off, D, idx=idx)
    assert device_status() == binding.GEMM_ERR_INDEX
    assert torch.equal(D[:, keep], want[:, keep])
    assert (D[bad] == 0).all()


def check_weights(counts, front, behind, N, K, dtype, out, exact, pad=8):
    gen = torch.Generator().manual_seed(N + K)
    M = front + sum(counts) + behind
    dD, A = wide(M, N, dtype, gen, exact=exact), wide(M, K, dtype, gen, exact=exact)
    e, ld = len(counts), (K + 7) // 8 * 8 + pad
    buf = torch.full((e, N + 1, ld), 7.0, dtype=ref.out_dtype(out), device="cuda")
    dB = buf[:, :N, :K]
    got = binding.gemm_grouped_weights(dD, A, offsets_of(counts, front), dB, alpha=2.0, out=out)
    assert got is dB
    what = (counts, N, K, dtype, out, pad)
    host = buf.cpu().float()
    assert (host[:, N:] == 7).all() and (host[:, :, K:] == 7).all(), what
    d, a = dD.cpu().double(), A.cpu().double()
    for g, (lo, hi) in enumerate(bounds(counts, front)):
        want = 2.0 * d[lo:hi].T @ a[lo:hi]
        if exact:
            assert torch.equal(dB[g].cpu(), want.float().to(ref.out_dtype(out))), (g, what)
        else:
            t = d[lo:hi].abs().T @ a[lo:hi].abs()
            b = 2.0 * sum_bound(hi - lo, out) * t + 2.0 ** -23 * want.abs()
            assert_close(dB[g], want, b + ref.rounding(want.abs() + b, out), (g, what))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("groups", GROUPS)
def test_weights_exact(form, groups):
    binding.gemm_debug_force_tile(*FORMS[form])
    counts, front, behind = GROUPS[groups]
    for i, (N, K) in enumerate(((1, 1), (70, 64), (129, 264), (300, 31))):
        check_weights(counts, front, behind, N, K, *KINDS[i % 3], True, pad=(8, 0, 3)[i % 3])


@pytest.mark.parametrize("form", FORMS)
def test_weights_every_remainder(form):
    """Groups whose last block of 64 rows holds 0 to 63 of them, over one and several stages."""
    binding.gemm_debug_force_tile(*FORMS[form])
    check_weights(list(range(65)), 1, 0, 72, 136, BF16, OUT_F32, True)
    check_weights([64 * 7 + r for r in range(0, 64, 5)], 0, 3, 72, 136, F16, OUT_F32, True)


@pytest.mark.parametrize("counts,N,K", [([700, 3, 0, 900], 777, 1000), ([2, 1, 0, 1] * 8, 1030, 520),
                                        ([400, 0, 1900, 20], 264, 328)])
def test_weights_normal(counts, N, K):
    for dtype, out in ((BF16, OUT_BF16), (F16, OUT_F32)):
        check_weights(counts, 2, 5, N, K, dtype, out, False)


def test_weights_without_rows():
    dB = torch.full((3, 24, 40), 7.0, device="cuda")
    binding.gemm_grouped_weights(torch.zeros(0, 24, dtype=F16, device="cuda"), torch.zeros(0, 40, dtype=F16, device="cuda"),
                                 torch.zeros(4, dtype=torch.int32, device="cuda"), dB)
    assert (dB == 0).all()


@pytest.mark.parametrize("form", FORMS)
def test_elements_past_32_bits(form):
    """Matrices of a stack and rows so far apart that element numbers do not fit 32 bits."""
    binding.gemm_debug_force_tile(*FORMS[form])
    gen = torch.Generator().manual_seed(3)
    counts, N, K, far = [30, 5, 45], 200, 136, (1 << 31) + 64
    off = offsets_of(counts, 0)
    big = torch.empty(2 * far + 300 * 512, dtype=F16, device="cuda")  # (8.6 GB)
    A, dD, small = wide(80, K, F16, gen), wide(80, N, F16, gen), stack(3, N, K, F16, gen, True)
    B = big.as_strided((3, N, K), (far, K, 1))
    B.copy_(small)
    want = binding.gemm_grouped(A, small, off), binding.gemm_grouped(dD, small, off, trans_b=True)
    assert torch.equal(binding.gemm_grouped(A, B, off), want[0])
    assert torch.equal(binding.gemm_grouped(dD, B, off, trans_b=True), want[1])
    wantB = binding.gemm_grouped_weights(dD, A, off, out=binding.OUT_F16)
    binding.gemm_grouped_weights(dD, A, off, B, out=binding.OUT_F16)
    assert torch.equal(B, wantB)
    pitch = 1 << 25  # (80 rows of it: 2^31 is passed at row 64)
    rows = big.as_strided((80, N), (pitch, 1))
    binding.gemm_grouped(A, small, off, rows, out=binding.OUT_F16)
    assert torch.equal(rows, want[0].half())
    rows = big.as_strided((80, K), (pitch, 1))
    rows.copy_(A)
    assert torch.equal(binding.gemm_grouped(rows, small, off), want[0])
    assert torch.equal(binding.gemm_grouped_weights(dD, rows, off, out=binding.OUT_F16), wantB)


def test_weights_of_one_row_far_apart():
    gen = torch.Generator().manual_seed(3)
    far, off = (1 << 31) + 8, offsets_of([30, 5, 45], 0)
    A, dD, small = wide(80, 136, F16, gen), wide(80, 1, F16, gen), stack(3, 1, 136, F16, gen, True)
    B = torch.empty(2 * far + 136, dtype=F16, device="cuda").as_strided((3, 1, 136), (far, far, 1))
    B.copy_(small)
    assert torch.equal(binding.gemm_grouped(A, B, off), binding.gemm_grouped(A, small, off))
    want = binding.gemm_grouped_weights(dD, A, off, out=binding.OUT_F16)
    binding.gemm_grouped_weights(dD, A, off, B, out=binding.OUT_F16)
    assert torch.equal(B, want)


def test_gradients_against_differences():
    """dA and dB of sum(dD * D) against central differences of the product itself, which is linear in
    each operand: on quarter-integers both are exact."""
    gen = torch.Generator().manual_seed(9)
    counts, N, K = [5, 0, 30], 24, 16
    M, off = sum(counts), offsets_of(counts, 0)
    A, B, dD = wide(M, K, F16, gen, exact=True), stack(3, N, K, F16, gen, True), wide(M, N, F16, gen, exact=True)
    dA = binding.gemm_grouped(dD, B, off, trans_b=True)
    dB = binding.gemm_grouped_weights(dD, A, off)
    loss = lambda a, b: (dD.double() * binding.gemm_grouped(a, b, off).double()).sum().item()  # noqa: E731
    for i, k in ((0, 0), (4, 15), (5, 3), (34, 8)):
        up, down = A.clone(), A.clone()
        up[i, k] += 0.25
        down[i, k] -= 0.25
        assert (loss(up, B) - loss(down, B)) / 0.5 == dA[i, k].item()
    for g, n, k in ((0, 0, 0), (1, 5, 5), (2, 23, 15)):
        up, down = B.clone(), B.clone()
        up[g, n, k] += 0.25
        down[g, n, k] -= 0.25
        assert (loss(A, up) - loss(A, down)) / 0.5 == dB[g, n, k].item()


# ---------------------------------------------------------------- rows by group

@pytest.mark.parametrize("M,E,choices", [(0, 3, 1), (1, 1, 1), (32, 8, 2), (33, 8, 1), (1000, 0, 1), (1024, 7, 1), (1025, 1024, 1), (1030, 3, 2),
                                         (16384, 64, 2), (65536, 256, 4), (65537, 5, 1), (131072, 1000, 2), (131073, 5, 1), (200000, 1024, 2),
                                         (3000000, 17, 1)])
def test_group_rows(M, E, choices):
    gen = torch.Generator().manual_seed(M + E)
    ids = torch.randint(-1, E + 2, (M,), generator=gen).int()
    if M > 100:
        ids[50:90] = 0  # (a run of one id)
        ids[7], ids[8] = -(1 << 31), (1 << 31) - 1
    given = ids.cuda() if choices == 1 else ids[:M // choices * choices].reshape(-1, choices).cuda()
    offsets, order, rows = binding.gemm_group_rows(given, E)
    flat = given.flatten().cpu().long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    want = torch.sort(key, stable=True).indices
    assert torch.equal(order.cpu().long(), want)
    assert torch.equal(rows.cpu().long(), want // choices)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(offsets.cpu().long(), torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0))))


def test_group_rows_without_rows_output():
    ids = torch.tensor([2, 0, 2, 1, 0], dtype=torch.int32, device="cuda")
    off, order = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (4, 5))
    st = binding.load_library().gemm_group_rows(5, 3, 1, ids.data_ptr(), off.data_ptr(), order.data_ptr(), None,
                                                torch.cuda.current_stream().cuda_stream)
    assert st == binding.GEMM_OK
    assert order.tolist() == [1, 4, 3, 0, 2] and off.tolist() == [0, 2, 3, 5]
