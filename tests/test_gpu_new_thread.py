"""Calls from a host thread that has not used the GPU before (needs a GB300)."""
import threading

import pytest
import torch

from gpu_helpers import DEV, device_status
from tensor_core_gemm_02_gb300 import binding

pytestmark = pytest.mark.gpu


def _in_new_thread(fn):
    got = []

    def body():
        try:
            got.append(fn())
        except Exception as e:  # noqa: BLE001 -- raised below
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join(timeout=120)
    assert not t.is_alive()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def _quarters(seed, rows, cols):
    r = torch.Generator().manual_seed(seed)
    return (torch.randint(-4, 5, (rows, cols), generator=r).float() / 4).to(torch.bfloat16).to(DEV)


def _operands(seed):
    return _quarters(seed, 256, 264), _quarters(seed + 1, 200, 264)


def _fp4(x):
    q, s = binding.gemm_quantize_e2m1(x[:, :256])
    return q, s


# each: operands in hand -> a call that writes D
CALLS = {
    "plain": lambda A, B: lambda D: binding.gemm_bf16(A, B, None, D),
    "few rows": lambda A, B: lambda D: binding.gemm_bf16(A[:16], B, None, D[:16]),
    "trans": lambda A, B: lambda D: binding.gemm_trans(A, B, None, D),
    "trans stored": lambda A, B: (lambda Bt: lambda D: binding.gemm_trans(A, Bt, None, D, trans_b=True))(B.t().contiguous()),
    "gated": lambda A, B: lambda D: binding.gemm_gated(A, B, B, D, act="relu"),
    "gated FP4": lambda A, B: (lambda a, b: lambda D: binding.gemm_gated_e2m1(*a, *b, *b, D, act="relu"))(_fp4(A), _fp4(B)),
    "quantiser": lambda A, B: lambda D: binding.gemm_quantize_e2m1(D[:, :192], Y=D[:, :192]),
}
KEPT = []  # (no address comes up twice: descriptors of earlier calls must not help)


@pytest.mark.parametrize("name", CALLS)
def test_first_call_of_a_thread(name):
    """The thread's first use of the GPU is the library's call, on operands not seen before."""
    A, B = _operands(1)
    outs = [torch.zeros((256, 200), device=DEV) for _ in range(2)]
    KEPT.extend([A, B, *outs])
    call = CALLS[name](A, B)
    torch.cuda.synchronize()
    _in_new_thread(lambda: call(outs[0]))
    call(outs[1])
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    assert name == "quantiser" or outs[0].abs().sum() > 0
    assert _in_new_thread(binding.gemm_check_device_status) == binding.GEMM_OK
    assert device_status() == binding.GEMM_OK
