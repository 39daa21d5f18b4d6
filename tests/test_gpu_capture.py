"""Calls captured into CUDA graphs and the buffers the library keeps for them (needs a GB300).

Quarter-integer inputs: every sum is exact in float32, so a replay's result is compared
bit for bit with the 64-bit form.
"""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import gated_ref as ref
from gated_ref import wide
from gpu_helpers import device_status
from tensor_core_gemm_02_gb300 import binding

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _clean():
    assert device_status() == binding.GEMM_OK
    yield
    assert device_status() == binding.GEMM_OK


def gen(seed):
    return torch.Generator().manual_seed(seed)


def exact(rows, cols, seed):
    return wide(rows, cols, BF16, gen(seed), exact=True)


class TransParts:
    """gemm_trans, the sum in parts."""

    def __init__(self, size):
        self.M, self.N, self.K = 100 * size, 130 * size, 4104
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert binding.gemm_query_plan(self.M, self.N, self.K, trans=(True, True), sm_count=sms).splits > 1
        self.x = [exact(self.K, self.M, 1), exact(self.K, self.N, 2)]
        self.out = [torch.empty((self.M, self.N), device="cuda")]

    def call(self):
        binding.gemm_trans(*self.x, None, self.out[0], trans_a=True, trans_b=True)

    def want(self):
        a, b = (t.cpu().double() for t in self.x)
        return [(a.T @ b).float()]


class Backward:
    """gemm_gated_backward, relu: few weights and many tokens, whose sums come in parts."""

    def __init__(self, size):
        M, N, K = (4104 if size == 1 else 8200), 64 * size, 72 * size
        self.x = [exact(M, N, 1), exact(M, N, 2), exact(M, N, 3), exact(M, K, 4), exact(N, K, 5), exact(N, K, 6)]
        new = lambda r, c, t=torch.float32: torch.empty((r, c), dtype=t, device="cuda")  # noqa: E731
        self.out = [new(M, K), new(N, K), new(N, K), new(M, N, BF16), new(M, N, BF16)]

    def call(self):
        dA, dBg, dBu, dG, dU = self.out
        binding.gemm_gated_backward(*self.x, dG=dG, dU=dU, dA=dA, dBg=dBg, dBu=dBu, act="relu")

    def want(self):
        dD, G, U, A, Bg, Bu = (t.cpu().double() for t in self.x)
        dG, dU = dD * U * (G > 0), dD * G.clamp(min=0)  # products of quarters: exact in bf16
        return [(dG @ Bg + dU @ Bu).float(), (dG.T @ A).float(), (dU.T @ A).float(), dG.bfloat16(), dU.bfloat16()]


class Skinny:
    """gemm_gated with few rows: parts of tiles in the stream-K workspace."""

    def __init__(self, size):
        assert binding.gemm_query_plan(16, 1500 * size, 2048, gated="16", sm_count=152).splits > 1
        self.x = [exact(16, 2048, 1), exact(1500 * size, 2048, 2), exact(1500 * size, 2048, 3)]
        self.out = [torch.empty((16, 1500 * size), device="cuda")]

    def call(self):
        binding.gemm_gated(*self.x, *self.out, act="relu")

    def want(self):
        return [ref.gated64(*self.x, "relu")[0].float()]


class FP4:
    """gemm_gated_e2m1 with scale rows not 16 bytes apart, which are copied first."""

    def __init__(self, size):
        M, N, K = 130, 70 * size, 64
        r, self.x = gen(1), []
        for rows in (M, N, N):
            self.x.append(torch.randint(0, 256, (rows, K // 2), generator=r, dtype=torch.uint8).cuda())
            scales = torch.full((K // 32, rows + 1), 127, dtype=torch.uint8)
            scales[:, 1:] = torch.randint(126, 129, (K // 32, rows), generator=r, dtype=torch.uint8)
            self.x.append(scales.cuda()[:, 1:])
        self.out = [torch.empty((M, N), device="cuda")]

    def call(self):
        binding.gemm_gated_e2m1(*self.x, *self.out, act="relu")

    def want(self):
        levels = torch.tensor([*ref.LEVELS, *-ref.LEVELS], dtype=torch.float64)

        def values(q, s):
            q, s = q.cpu(), s.cpu()
            codes = torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1)
            return levels[codes.long()] * torch.exp2(s.double() - 127).T.repeat_interleave(32, dim=1)

        return [ref.gated64(*(values(*self.x[i:i + 2]) for i in (0, 2, 4)), "relu")[0].float()]


FORMS = [TransParts, Backward, Skinny, FP4]


def check(form, what):
    for i, (got, want) in enumerate(zip(form.out, form.want())):
        assert torch.equal(got.cpu(), want), (what, i)


@pytest.mark.parametrize("form", FORMS)
def test_replay_after_a_larger_call(form):
    """The buffers that a graph's calls were captured with stay theirs when a larger call on the
    stream needs larger ones, and memory allocated after that is not written."""
    s = torch.cuda.Stream()
    small = form(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        small.call()
    graph.replay()
    torch.cuda.synchronize()
    check(small, "replay")
    large = form(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        large.call()
    s.synchronize()
    check(large, "larger call")
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for t in small.x[:1]:
        t.mul_(-1) if t.dtype == BF16 else t.bitwise_xor_(0x88)  # other inputs (signs)
    for t in small.out:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check(small, "replay after a larger call")
    assert all(bool((t == 7).all()) for t in others)
    with torch.cuda.stream(s):
        large.call()
    s.synchronize()
    check(large, "larger call after replays")


@pytest.mark.parametrize("form", [f.__name__ for f in FORMS])
def test_first_call_inside_a_capture(form):
    """A process's first call of the library may be a captured one; the same stream's calls and
    replays after it are right as well."""
    code = textwrap.dedent(f"""
        import sys, torch
        sys.path[:0] = {[os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]!r}
        import test_gpu_capture as t
        form = t.{form}(1)
        torch.cuda.synchronize()
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            form.call()
        for _ in range(2):
            with torch.cuda.stream(s):
                form.call()
            s.synchronize()
            t.check(form, "call")
            [x.zero_() for x in form.out]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            t.check(form, "replay")
        assert t.device_status() == t.binding.GEMM_OK
        print("right")
        """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("right"), r.stdout + r.stderr
