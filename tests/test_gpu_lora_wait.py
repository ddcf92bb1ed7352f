"""The time-out path of the adapters' tensor-core kernels, run on the GPU
without a fault: a test build sends the first wait of the MMA warp to an mbarrier
that nothing arrives on (a 200 us limit).  shrink reports 0x401, the gradients'
kernel 0x402, expand 0x403; no drain runs out, and the context stays usable."""

from __future__ import annotations

import ctypes

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding, build

pytestmark = pytest.mark.gpu

SHRINK_WAIT, GRAD_WAIT, EXPAND_WAIT = 0x401, 0x402, 0x403


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64)]


def rows(t):
    return ctypes.byref(Rows(t.data_ptr(), t.stride(0), t.stride(1)))


@pytest.mark.parametrize("B,S,K,N,R,NA", [(2, 100, 1536, 72, 16, 1), (3, 40, 64, 200, 64, 2)])
def test_waits_that_run_out_report_and_return(B, S, K, N, R, NA):
    lib()
    L = ctypes.CDLL(build.build(extra_flags=build.WAIT_TEST_FLAGS, variant="waittest"))
    for n in ("adaln_lora_fwd", "adaln_lora_bwd"):
        getattr(L, n).argtypes = binding._SIGNATURES[n][1]
    gen = torch.Generator("cuda").manual_seed(0)
    t = torch.bfloat16
    x, g = (torch.randn((B, S, C), generator=gen, device="cuda").to(t) for C in (K, N))
    A, U = (torch.randn((NA, R, C), generator=gen, device="cuda").to(t) for C in (K, N))
    scale, ids = torch.ones(NA, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        out, state = binding.adaln_lora_fwd(x, A, U, scale, ids)
        return (out, state, *binding.adaln_lora_bwd(g, x, state, A, U, scale, ids))
    before = step()
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    out, state, dx, dA, dU = (torch.empty_like(v) for v in before)
    st = torch.cuda.current_stream().cuda_stream
    w = (A.data_ptr(), U.data_ptr(), scale.data_ptr(), ids.data_ptr(), 0, None)
    assert L.adaln_lora_fwd(rows(x), *w, None, rows(out), state.data_ptr(), state.numel(), B, S, K, N, R, NA, st) == 0
    assert L.adaln_device_error() == SHRINK_WAIT
    ws = torch.zeros(binding.adaln_lora_bwd_workspace_bytes(B, S, K, N, R), dtype=torch.uint8, device="cuda")
    # only dU: the gradients' kernel alone
    assert L.adaln_lora_bwd(rows(g), rows(x), before[1].data_ptr(), *w, None, None, None, dU.data_ptr(), 0,
                            ws.data_ptr(), ws.numel(), B, S, K, N, R, NA, st) == 0
    assert L.adaln_device_error() == GRAD_WAIT
    # samples without an adapter: shrink has nothing to wait for, expand copies y
    none = (*w[:3], torch.full_like(ids, -1), *w[4:])
    y = torch.zeros_like(out)
    assert L.adaln_lora_fwd(rows(x), *(v.data_ptr() if torch.is_tensor(v) else v for v in none), rows(y), rows(out),
                            state.data_ptr(), state.numel(), B, S, K, N, R, NA, st) == 0
    assert L.adaln_device_error() == EXPAND_WAIT
    assert L.adaln_device_error() == 0
    after = step()
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(after[2:], before[2:]))
    assert torch.equal(after[0].view(torch.uint8), before[0].view(torch.uint8))
