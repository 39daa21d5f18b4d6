"""The operators for layers of experts together, as they are used (needs a GB300): the example's
layer against autograd in 64 bits, captured steps, threads, streams, first calls, time-outs."""
import os
import subprocess
import sys
import textwrap
import threading

import pytest
import torch

from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import experts  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
FORMS = {"auto": (0, 0), "few": (2, 0), "single64": (1, 64), "single128": (1, 128), "single256": (1, 256), "pair256": (3, 256)}


@pytest.fixture(autouse=True)
def _clean():
    binding.gemm_debug_force_tile(0, 0)
    assert device_status() == binding.GEMM_OK
    yield
    binding.gemm_debug_force_tile(0, 0)
    binding.gemm_debug_inject(0)
    binding.gemm_set_wait_timeout(0)
    assert device_status() == binding.GEMM_OK


def relative(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("tokens,choices", [(300, 2), (5, 3)])
def test_layer_against_autograd(tokens, choices):
    """Forward and every gradient against autograd on the same 16-bit weights in 64 bits.  Each path
    has at most six roundings to float16 (G, U, H, dO, dG or dU, and dH's products of those), each at
    most 2^-11 of what it rounds, and products of whole matrices do not grow relative errors of their
    operands beyond a small factor: 2^-11 x 6 x 4 in the Frobenius norm."""
    gen = torch.Generator().manual_seed(tokens)
    layer = experts.Experts(6, 136, 72, dtype=F16, seed=3)
    X = torch.randn((tokens, 136), generator=gen).half()
    scores = torch.randn((tokens, 6), generator=gen)
    scores[:, 4] = -9.0  # an expert nobody chooses
    ids, w = experts.route(scores, choices)
    dY = torch.randn((tokens, 136), generator=gen)
    Y, kept = layer.forward(X.cuda(), ids.cuda(), w.cuda())
    dX, dw, grads = layer.backward(dY.cuda(), kept)
    x, wt = X.double().requires_grad_(), w.double().requires_grad_()
    W = {k: getattr(layer, k).cpu().double().requires_grad_() for k in ("Wg", "Wu", "Wd")}
    want = torch.zeros_like(x)
    rows = []
    for t in range(tokens):
        y = 0
        for j in range(choices):
            e = int(ids[t, j])
            h = torch.nn.functional.silu(W["Wg"][e] @ x[t]) * (W["Wu"][e] @ x[t])
            y = y + wt[t, j] * (W["Wd"][e] @ h)
        rows.append(y)
    want = torch.stack(rows)
    want.backward(dY.double())
    tol = 2.0 ** -11 * 6 * 4
    assert relative(Y, want.detach()) < tol
    assert relative(dX, x.grad) < tol and relative(dw, wt.grad) < tol
    for k, g in grads.items():
        assert relative(g, W[k].grad) < tol, k
        assert (g[4] == 0).all()


def test_example_runs():
    losses = experts.run(tokens=200, model=128, hidden=64, experts=5, steps=3, say=lambda s: None)
    assert len(losses) == 3 and all(x == x for x in losses)


# ---------------------------------------------------------------- graphs, streams, threads

def quarters(shape, seed, dtype=BF16):
    r = torch.Generator().manual_seed(seed)
    return (torch.randint(-4, 5, shape, generator=r).float() / 4).to(dtype).cuda()


def test_captured_step_follows_other_assignments():
    """Grouping, products and gradients in one graph, replayed on other ids: the offsets are read on
    the device.  On a stream that is not the current one's; nothing of the last replay remains."""
    E, T, N, K = 7, 90, 72, 136
    X, B, dD = quarters((T, K), 1), quarters((E, N, K), 2), quarters((2 * T, N), 3)
    ids = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    order, rows = (torch.zeros(2 * T, dtype=torch.int32, device="cuda") for _ in range(2))
    D, dA, dB = torch.zeros((2 * T, N), device="cuda"), torch.zeros((2 * T, K), device="cuda"), torch.zeros((E, N, K), device="cuda")
    Xs = torch.zeros((2 * T, K), dtype=BF16, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def step():
        binding.gemm_group_rows(ids, E, off, order, rows)
        binding.gemm_grouped(X, B, off, D, idx=rows)
        binding.gemm_grouped(dD, B, off, dA, trans_b=True)
        torch.index_select(X, 0, rows, out=Xs)
        binding.gemm_grouped_weights(dD, Xs, off, dB)

    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in range(4):
        new = torch.randint(0, E if seed else 1, (T, 2), generator=torch.Generator().manual_seed(seed)).int()
        new[new == 3] = -1  # (dropped: of no group)
        ids.copy_(new)
        D.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        flat = new.flatten().long()
        key = torch.where(flat < 0, E, flat)
        at = torch.sort(key, stable=True).indices
        want = torch.full((2 * T, N), 7.0, dtype=torch.float64)
        wantA = torch.zeros((E, N, K), dtype=torch.float64)
        x, b, d = X.cpu().double(), B.cpu().double(), dD.cpu().double()
        for i, a in enumerate(at):
            e = int(key[a])
            if e < E:
                want[i] = x[a // 2] @ b[e].T
                wantA[e] += torch.outer(d[i], x[a // 2])
        assert torch.equal(D.cpu().double(), want), seed
        assert torch.equal(dB.cpu().double(), wantA), seed


def test_two_graphs_of_two_streams_share_nothing():
    """Graphs captured on two streams, replayed at once, keep their own workspaces."""
    X = [torch.randn((3, 300, 200 + 8 * i), device="cuda") for i in range(2)]
    Y = [torch.empty_like(x) for x in X]
    want = [binding.gemm_orthogonalize(x) for x in X]
    streams = [torch.cuda.Stream() for _ in X]
    graphs = [torch.cuda.CUDAGraph() for _ in X]
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            binding.gemm_orthogonalize(X[i], Y[i])
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(Y[i], want[i])


def test_replay_after_a_larger_call():
    """A graph's workspace stays its own when a larger call on its stream needs a larger one."""
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    X, L = torch.randn((2, 130, 100), device="cuda"), torch.randn((4, 700, 900), device="cuda")
    ids = torch.randint(0, 50, (140000,), dtype=torch.int32, device="cuda")
    more = torch.randint(0, 900, (400000,), dtype=torch.int32, device="cuda")
    Y, want = torch.empty_like(X), binding.gemm_orthogonalize(X)
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (51, 140000, 140000)]
    wanted = binding.gemm_group_rows(ids, 50)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        binding.gemm_orthogonalize(X, Y)
        binding.gemm_group_rows(ids, 50, *outs)
    with torch.cuda.stream(s):
        binding.gemm_orthogonalize(L)
        binding.gemm_group_rows(more, 900)
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for _ in range(3):
        Y.zero_()
        [o.zero_() for o in outs]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        assert all(torch.equal(a, b) for a, b in zip(outs, wanted))
    assert all(bool((t == 7).all()) for t in others)


@pytest.mark.parametrize("raw", [False, True])
def test_a_stream_that_is_not_the_current_one(raw):
    """Every step of a call, a new output's zeros too, is on the stream it is given, whatever else the
    current one still has to do."""
    A, B, dD = quarters((150, 136), 1), quarters((3, 200, 136), 2), quarters((150, 200), 3)
    ids = torch.randint(-1, 3, (150,), dtype=torch.int32, device="cuda")
    off = binding.gemm_group_rows(ids, 3)[0]
    calls = [lambda **k: binding.gemm_group_rows(ids, 3, **k)[1], lambda **k: binding.gemm_grouped(A, B, off, **k),
             lambda **k: binding.gemm_grouped(dD, B, off, trans_b=True, out=binding.OUT_BF16, **k),
             lambda **k: binding.gemm_grouped_weights(dD, A, off, **k), lambda **k: binding.gemm_orthogonalize(B, **k)]
    want = [c() for c in calls]
    s, busy = torch.cuda.Stream(), torch.empty(1 << 31, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):
        busy.fill_(1)
    got = [c(stream=s.cuda_stream if raw else s) for c in calls]
    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream_and_memory_still_in_use(raw):
    """The current stream has still to write blocks of the outputs' sizes when they are freed: the
    outputs of a call on another stream are not laid there."""
    A, B, dD = quarters((150, 136), 1), quarters((3, 200, 136), 2), quarters((150, 200), 3)
    ids = torch.randint(-1, 3, (150,), dtype=torch.int32, device="cuda")
    off = binding.gemm_group_rows(ids, 3)[0]
    calls = [lambda **k: binding.gemm_group_rows(ids, 3, **k)[1], lambda **k: binding.gemm_grouped(A, B, off, **k),
             lambda **k: binding.gemm_grouped(dD, B, off, trans_b=True, out=binding.OUT_BF16, **k),
             lambda **k: binding.gemm_grouped_weights(dD, A, off, **k), lambda **k: binding.gemm_orthogonalize(B, **k),
             lambda **k: binding.gemm_bf16(A, B[0], **k), lambda **k: binding.gemm_trans(dD, A, trans_a=True, trans_b=True, **k)]
    want = [c() for c in calls]
    s, busy = torch.cuda.Stream(), torch.empty(1 << 31, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):
        busy.fill_(1)
    freed = [torch.empty_like(w).fill_(99) for w in want for _ in range(8)]
    del freed
    got = [c(stream=s.cuda_stream if raw else s) for c in calls]
    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i
    assert torch.equal(calls[1](stream=0), want[1])


def _ortho(i):
    X = torch.randn((2, 100 + 40 * i, 150), device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
    return lambda: binding.gemm_orthogonalize(X)


def _sort(i):
    ids = torch.randint(0, 40 + i, (140000 + 1000 * i,), dtype=torch.int32, device="cuda")
    return lambda: binding.gemm_group_rows(ids, 40 + i)[1]


def _grouped(i):
    A, B = quarters((150 + i, 136), i), quarters((5, 200, 136), 9 + i)
    off = torch.tensor([0, 20 + i, 20 + i, 90, 91, 150], dtype=torch.int32, device="cuda")
    return lambda: binding.gemm_grouped(A, B, off)


@pytest.mark.parametrize("make", [_ortho, _sort, _grouped])
@pytest.mark.parametrize("one", [True, False])
def test_threads(make, one):
    """Threads that share a stream (and with it the kept buffers), or have one each: each result as
    alone, bit for bit."""
    calls = [make(i) for i in range(3)]
    want = [c().clone() for c in calls]
    shared = torch.cuda.Stream()
    torch.cuda.synchronize()
    go, failures = threading.Barrier(len(calls)), []

    def worker(i):
        try:
            s = shared if one else torch.cuda.Stream()
            with torch.cuda.stream(s):
                for it in range(4):
                    go.wait(timeout=60)
                    outs = [calls[i]() for _ in range(20)]
                    s.synchronize()
                    failures.extend((i, it, j) for j, o in enumerate(outs) if not torch.equal(o, want[i]))
        except Exception as e:  # noqa: BLE001 -- reported below
            failures.append((i, repr(e)))
            go.abort()

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not any(t.is_alive() for t in threads)
    assert not failures, failures[:5]


def _gathered(i):
    A, B = quarters((900, 520), i), quarters((4, 2056, 520), 9 + i)
    idx = torch.randint(0, 900, (3000 + 100 * i,), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 1500 + i, 1500 + i, 2200, 3000], dtype=torch.int32, device="cuda")
    return lambda: binding.gemm_grouped(A, B, off, idx=idx)


@pytest.mark.parametrize("one", [True, False])
def test_threads_with_gathered_rows(one):
    test_threads(_gathered, one)


def test_gathered_rows_replayed_after_a_larger_call():
    """The rows laid out in order are a graph's own: on two streams at once, and after a larger call."""
    calls = [_gathered(i) for i in range(2)]
    want = [c().clone() for c in calls]
    streams, graphs, got = [torch.cuda.Stream() for _ in calls], [torch.cuda.CUDAGraph() for _ in calls], []
    torch.cuda.synchronize()
    for c, s, g in zip(calls, streams, graphs):
        with torch.cuda.graph(g, stream=s):
            got.append(c())
    A, B = quarters((100, 2056), 5), quarters((1, 2056, 2056), 6)
    off = torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
    idx = torch.randint(0, 100, (9000,), dtype=torch.int32, device="cuda")
    with torch.cuda.stream(streams[0]):
        larger = binding.gemm_grouped(A, B, off, idx=idx)
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for _ in range(3):
        [t.zero_() for t in got]
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 7).all()) for t in others)
    assert torch.equal(larger, binding.gemm_grouped(A[idx.long()].contiguous(), B, off))


def test_gathered_rows_without_memory_for_them():
    """Where the workspace cannot be had the product gathers the rows itself: the same bits, also
    captured, and the calls after it have the workspace again.  (A stream of its own, which keeps
    none yet.)"""
    call, s, graph = _gathered(0), torch.cuda.Stream(priority=-1), torch.cuda.CUDAGraph()
    want, X = call().clone(), torch.randn((2, 300, 200), device="cuda")
    torch.cuda.synchronize()
    binding.gemm_debug_inject(2)
    with torch.cuda.stream(s):
        got = call()
        with pytest.raises(binding.GemmError):
            binding.gemm_orthogonalize(X)  # (which has no other way)
    with torch.cuda.graph(graph, stream=s):
        kept = call()
    binding.gemm_debug_inject(0)
    graph.replay()
    with torch.cuda.stream(s):
        again = call()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(kept, want) and torch.equal(again, want)


def test_memory_kept_for_gathered_rows():
    """A call of 5 GiB and one of 7.9 keep 8 GiB between them."""
    M, N = 1 << 20, 512
    idx = torch.randint(0, 50, (M,), dtype=torch.int32, device="cuda")
    off, D = torch.tensor([0, M], dtype=torch.int32, device="cuda"), torch.empty((M, N), dtype=BF16, device="cuda")
    operands = [(quarters((50, K), K), quarters((1, N, K), 1)) for K in (2560, 4032)]
    s, free = torch.cuda.Stream(priority=-1), []
    for A, B in operands:
        want = (A.double() @ B[0].double().T).to(BF16)[idx.long()]
        torch.cuda.synchronize()
        free.append(torch.cuda.mem_get_info()[0])
        binding.gemm_grouped(A, B, off, D, idx=idx, out=binding.OUT_BF16, stream=s)
        torch.cuda.synchronize()
        free.append(torch.cuda.mem_get_info()[0])
        assert torch.equal(D, want)
        del want
    taken = (free[0] - free[1]) + (free[2] - free[3])
    assert 7 << 30 < taken < (8 << 30) + (64 << 20), taken


@pytest.mark.parametrize("what", ["_ortho", "_sort", "_grouped"])
def test_first_call_of_a_process_inside_a_capture_on_a_new_thread(what):
    code = textwrap.dedent(f"""
        import sys, threading, torch
        sys.path[:0] = {[os.path.dirname(os.path.abspath(__file__)), ROOT]!r}
        import test_gpu_experts as t
        call, got = t.{what}(1), []
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got.append(call())
        thread = threading.Thread(target=lambda: got.append(call()))
        thread.start()
        thread.join()
        for _ in range(2):
            got[0].zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(*got)
        assert t.device_status() == t.binding.GEMM_OK
        print("right")
        """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("right"), r.stdout + r.stderr


def test_calls_one_behind_another():
    """Each reads what the call before it wrote, on one stream without a synchronisation between."""
    E, N, K = 5, 96, 96
    B = quarters((E, N, K), 4) / 4
    ids = torch.randint(0, E, (160,), generator=torch.Generator().manual_seed(2)).int()
    for i in range(20):
        given = ids.roll(i).cuda()
        off, order, rows = binding.gemm_group_rows(given, E)
        A = quarters((160, K), 50 + i)
        D = binding.gemm_grouped(A, B.to(BF16), off, idx=rows, out=binding.OUT_BF16)
        dB = binding.gemm_grouped_weights(D, D, off)
        Y = binding.gemm_orthogonalize(dB, steps=1)
        want = torch.stack([A[k].float() @ B[int(given[k])].float().T for k in rows.tolist()]).bfloat16()
        assert torch.equal(D, want), i
        for e in range(E):
            d = D[off[e]:off[e + 1]].double()
            assert (dB[e].double() - d.T @ d).abs().max() <= 1e-3 * (d.abs().T @ d.abs()).max() + 1e-6
        assert torch.equal(Y, binding.gemm_orthogonalize(dB, steps=1))


# ---------------------------------------------------------------- time-outs

def _timed_out(call):
    binding.gemm_set_wait_timeout(20_000_000)
    binding.gemm_debug_inject(1)
    call()
    assert device_status() == binding.GEMM_ERR_TIMEOUT
    binding.gemm_debug_inject(0)
    binding.gemm_set_wait_timeout(0)
    return call()


@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_runs_out(form):
    """A stage that never fills: the kernels give up, say so, and the next call works."""
    binding.gemm_debug_force_tile(*FORMS[form])
    A, B, dD = quarters((300, 328), 1), quarters((3, 264, 328), 2), quarters((300, 264), 3)
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    for out in (binding.OUT_F32, binding.OUT_BF16):
        want = binding.gemm_grouped(A, B, off, out=out)
        assert torch.equal(_timed_out(lambda: binding.gemm_grouped(A, B, off, out=out)), want)
        want = binding.gemm_grouped(dD, B, off, trans_b=True, out=out)
        assert torch.equal(_timed_out(lambda: binding.gemm_grouped(dD, B, off, trans_b=True, out=out)), want)
        want = binding.gemm_grouped_weights(dD, A, off, out=out)
        assert torch.equal(_timed_out(lambda: binding.gemm_grouped_weights(dD, A, off, out=out)), want)
    for dtype in (torch.float32, BF16):
        X = torch.randn((2, 300, 290), device="cuda").to(dtype)
        want = binding.gemm_orthogonalize(X, steps=1)
        assert torch.equal(_timed_out(lambda: binding.gemm_orthogonalize(X, steps=1)), want)


@pytest.mark.parametrize("out", [binding.OUT_F32, binding.OUT_BF16])
@pytest.mark.parametrize("counts,N", [([3, 0, 5, 1], 200), ([1] * 80, 8)])
def test_a_wait_that_runs_out_in_a_long_sum(counts, N, out):
    """Few rows, sums of many fills of the accumulators, on two CTAs a tile and on one."""
    A, B = quarters((sum(counts), 14336), 1), quarters((len(counts), N, 14336), 2)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    want = binding.gemm_grouped(A, B, off, out=out)
    assert torch.equal(_timed_out(lambda: binding.gemm_grouped(A, B, off, out=out)), want)
