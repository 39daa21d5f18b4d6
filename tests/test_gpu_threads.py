"""Concurrent calls from several host threads, each on a stream of its own (needs a GB300).

The library keeps per-device and per-stream state on the host (tensor-map cache,
stream-K workspaces and counters, dequantisation buffers) behind locks.  Four
threads run a mix of every kernel form at once, each on its own stream, many
times over; with exact inputs every result must equal, bit for bit, the one a
single-threaded call gives.
"""
import threading

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, device_status, run
from tensor_core_gemm_02_gb300 import binding, workloads
from tensor_core_gemm_02_gb300.workloads import OUT_BF16, OUT_F32

pytestmark = pytest.mark.gpu


def _fp4(seed, M, N, K):
    rng = np.random.default_rng(seed)
    A = torch.from_numpy((rng.integers(-4, 5, (M, K)) / 4).astype(np.float32)).to(torch.bfloat16)
    Bq = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8))
    Bs = torch.from_numpy(rng.integers(125, 130, (K // 32, N)).astype(np.uint8))
    C = torch.from_numpy((rng.integers(-4, 5, (M, N)) / 4).astype(np.float32))
    return workloads.Problem(f"fp4_{M}x{N}x{K}", A, Bq, C, alpha=0.5, beta=1.0, out=OUT_F32, Bs=Bs)


def _problems():
    q = dict(values="quarter")
    acc = workloads.random_problem(57, 16, 2048, 1024, dtype="bf16", with_c=True, alpha=-0.5, **q)
    return [
        # skinny stream-K (split tiles, last-arriver reduction)
        workloads.random_problem(51, 16, 4096, 2048, dtype="bf16", with_c=True, alpha=0.5, **q),
        # tile kernel, ragged
        workloads.random_problem(52, 300, 520, 264, dtype="f16", with_c=True, alpha=2.0,
                                 beta=0.5, out=OUT_BF16, **q),
        # gathered rows
        workloads.random_problem(53, 600, 2048, 512, dtype="bf16", with_c=True, alpha=0.5,
                                 gather_rows=333, **q),
        # scattered rows
        workloads.random_problem(54, 200, 300, 264, dtype="bf16", with_c=True, alpha=0.5,
                                 scatter_rows=700, **q),
        # FP4 weights (skinny form with converter warps)
        _fp4(55, 16, 2048, 1024),
        # dense 256 x 512 pair form
        workloads.random_problem(56, 1024, 2048, 2048, dtype="bf16", **q),
        # accumulate into float32 D (atomic adds; exact, so the order does not matter)
        workloads.Problem("acc", acc.A, acc.B, None, alpha=acc.alpha, beta=0.0, out=OUT_F32,
                          D0=acc.C, accumulate=True),
    ]


def test_threads_on_own_streams_match_single_threaded():
    problems = _problems()
    want = [run(p).cpu() for p in problems]
    torch.cuda.synchronize()
    failures = []

    def worker(tid):
        try:
            s = torch.cuda.Stream(device=DEV)
            with torch.cuda.stream(s):
                for it in range(8):
                    outs = [run(p, stream=s) for p in problems]
                    s.synchronize()
                    for k, (got, ref) in enumerate(zip(outs, want)):
                        if not torch.equal(got.cpu(), ref):
                            failures.append((tid, it, problems[k].name))
        except Exception as e:  # noqa: BLE001 -- reported below
            failures.append((tid, -1, repr(e)))

    threads = [threading.Thread(target=worker, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not any(t.is_alive() for t in threads)
    assert not failures, failures[:5]
    assert device_status() == binding.GEMM_OK


def _quarters(seed, rows, cols):
    r = torch.Generator().manual_seed(seed)
    return (torch.randint(-4, 5, (rows, cols), generator=r).float() / 4).to(torch.bfloat16).to(DEV)


def _trans_parts(i):
    """gemm_trans in parts, another shape per thread."""
    M, N, K = 128 + 32 * i, 64 + 8 * i, 4096
    A, B = _quarters(60 + i, K, M), _quarters(70 + i, K, N)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert binding.gemm_query_plan(M, N, K, trans=(True, True), sm_count=sms).splits > 1
    return lambda s: binding.gemm_trans(A, B, trans_a=True, trans_b=True, stream=s)


def test_bare_calls_from_threads_on_one_stream():
    """As below for gemm_trans in parts, through the C entry with its arguments in hand: the calls'
    two launches are as close to one another's as they get."""
    s, lib = torch.cuda.Stream(device=DEV), binding.load_library()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    operands, want, outs, calls = [], [], [], []
    for i in range(4):
        M, N, K = 128 + 32 * i, 64 + 8 * i, 4096
        A, B = _quarters(60 + i, K, M), _quarters(70 + i, K, N)
        assert binding.gemm_query_plan(M, N, K, trans=(True, True), sm_count=sms).splits > 1
        operands.append((A, B))
        want.append((A.double().T @ B.double()).float())
        outs.append(torch.zeros((200, M, N), device=DEV))
        calls.append([(M, N, K, 1, 1, A.data_ptr(), M, 1, B.data_ptr(), N, None, 0, D.data_ptr(), N, OUT_F32,
                       1.0, 0.0, s.cuda_stream) for D in outs[i]])
    torch.cuda.synchronize()
    go, status = threading.Barrier(len(calls)), []

    def worker(i):
        binding.gemm_check_device_status(s)
        for _ in range(10):
            go.wait(timeout=60)
            status.extend({lib.gemm_trans(*args) for args in calls[i]})

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not any(t.is_alive() for t in threads) and set(status) == {binding.GEMM_OK}
    s.synchronize()
    for i, D in enumerate(outs):
        wrong = [j for j in range(len(D)) if not torch.equal(D[j], want[i])]
        assert not wrong, (i, wrong[:8], len(wrong))
    assert device_status() == binding.GEMM_OK


def _gradients_in_parts(i):
    M, N, K = 4096, 64 + 16 * i, 72 + 8 * i
    dD, G, U, A = (_quarters(80 + 10 * i + j, M, n) for j, n in enumerate((N, N, N, K)))
    Bg, Bu = _quarters(84 + 10 * i, N, K), _quarters(85 + 10 * i, N, K)
    return lambda s: torch.cat([t.flatten() for t in binding.gemm_gated_backward(
        dD, G, U, A, Bg, Bu, act="relu", stream=s)[:3]])


def _weights_to_bf16(i):
    """FP4 weights and many rows: the weights are converted into a buffer first."""
    p = _fp4(90 + i, 200, 256 + 32 * i, 512)
    A, B, Bs = p.A.to(DEV), p.B.to(DEV), p.Bs.to(DEV)
    return lambda s: binding.gemm_bf16_e2m1(A, B, Bs, stream=s)


def _copied_scales(i, few=False):
    """Both operands FP4, scale rows not 16 bytes apart (copied into buffers first)."""
    M, N, K = 16 if few else 200, 256 + 32 * i, 512
    r = torch.Generator().manual_seed(100 + i)
    x = []
    for rows in (M, N, N):
        x.append(torch.randint(0, 256, (rows, K // 2), generator=r, dtype=torch.uint8).to(DEV))
        x.append(torch.randint(126, 129, (K // 32, rows + 1), generator=r, dtype=torch.uint8).to(DEV)[:, 1:])
    return lambda s: binding.gemm_gated_e2m1(*x, act="relu", stream=s)


def _copied_scales_few(i):
    return _copied_scales(i, few=True)


def _weight_scales(i):
    """FP4 weights and few rows, the same of their scales."""
    p = _fp4(110 + i, 16, 2048 + 64 * i, 512)
    A, B = p.A.to(DEV), p.B.to(DEV)
    Bs = torch.cat((p.Bs[:, :1], p.Bs), dim=1).to(DEV)[:, 1:]
    return lambda s: binding.gemm_bf16_e2m1(A, B, Bs, stream=s)


def _plain_e2m1(i):
    M, N, K = 200, 256 + 32 * i, 512
    r = torch.Generator().manual_seed(120 + i)
    x = []
    for rows in (M, N):
        x.append(torch.randint(0, 256, (rows, K // 2), generator=r, dtype=torch.uint8).to(DEV))
        x.append(torch.randint(126, 129, (K // 32, rows + 1), generator=r, dtype=torch.uint8).to(DEV)[:, 1:])
    return lambda s: binding.gemm_e2m1(*x, stream=s)


@pytest.mark.parametrize("make", [_trans_parts, _gradients_in_parts, _weights_to_bf16, _copied_scales,
                                  _copied_scales_few, _weight_scales, _plain_e2m1])
def test_threads_on_one_stream(make):
    """Calls of several launches that pass data on through a kept buffer, from threads that share one
    stream: each result as alone, bit for bit (exact sums)."""
    s = torch.cuda.Stream(device=DEV)
    calls = [make(i) for i in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = [call(s).clone() for call in calls]
    s.synchronize()
    go, failures = threading.Barrier(len(calls)), []

    def worker(i):
        try:
            with torch.cuda.stream(s):
                for it in range(6):
                    go.wait(timeout=60)
                    outs = [calls[i](s) for _ in range(50)]
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
    assert device_status() == binding.GEMM_OK
