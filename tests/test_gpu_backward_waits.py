"""A wait that runs out in the training kernels: the kernel returns, the status
word says so, and the next ordinary call in the same context gives the same
bits as one before."""
import pytest
import torch

import grouped_expert_gemm_router_b200 as moe
from test_gpu_backward import CASES, Layer

pytestmark = pytest.mark.gpu

# more units than SMs (each CTA has several), a reduction longer than the ring of stages
LONG = (2000, 512, 2048, 16, 2, None, "uniform")


def _checkpoint(L, shape, out):
    moe.moe_grouped_swiglu_checkpoint(shape, L.x_perm, L.w_gate, L.w_up, *out, L.ws)


def _down(L, shape, out):
    moe.moe_grouped_down_backward(shape, L.dy, L.w_down, L.ck["g_q"], L.ck["u_q"], L.ck["scale"], *out, L.ws)


def _swiglu(L, shape, out):
    moe.moe_grouped_swiglu_backward(shape, L.dg, L.du, L.w_gate, L.w_up, *out, L.ws)


def _buffers(L, op):
    if op is _checkpoint:
        ck = moe.alloc_checkpoint(L.shape)
        return [L.poison(L.P, L.F)] + [ck[n].fill_(0) for n in ("g_q", "u_q", "scale")]
    return [L.poison(L.P, L.F) for _ in range(3)] if op is _down else [L.poison(L.P, L.H)]


def _bits(out):
    return [t.view(torch.uint8) for t in out]


@pytest.mark.parametrize("op", [_checkpoint, _down, _swiglu], ids=["checkpoint", "down", "swiglu"])
@pytest.mark.parametrize("case", ["two_tiles", "capacity", "wide_units", "long"])
def test_wait_of_a_training_gemm_expires_and_reports(case, op):
    """CTA 0's token producer never loads its first stage."""
    L = Layer(case, case=LONG if case == "long" else CASES[case])
    L.dy, L.dg, L.du, L.ck = L.rows(L.P, L.H), L.rows(L.P, L.F), L.rows(L.P, L.F), L.checkpoint()
    ref = _buffers(L, op)
    op(L, L.shape, ref)
    assert L.status() == 0
    s = L.shape
    stall = moe.make_shape(s.T, s.H, s.F, s.E, s.k, C=s.C, flags=s.flags | moe.MOE_FLAG_TEST_STALL_GEMM)
    moe.moe_set_wait_timeout_ns(50_000_000)
    try:
        op(L, stall, _buffers(L, op))
        status = moe.moe_read_status(L.ws, clear=True)
    finally:
        moe.moe_set_wait_timeout_ns(1_000_000_000)
    assert status == moe.MOE_DEV_GEMM_TIMEOUT, hex(status)
    got = _buffers(L, op)
    op(L, s, got)
    assert L.status() == 0
    for a, b in zip(_bits(got), _bits(ref)):
        assert torch.equal(a, b)
