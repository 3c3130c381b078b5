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


def _gate_up_wgrad(L, shape, out):
    moe.moe_grouped_swiglu_wgrad(shape, L.x_perm, L.dg, L.du, *out, L.ws)


def _down_wgrad(L, shape, out):
    moe.moe_grouped_down_wgrad(shape, L.h, L.dy, *out, L.ws)


# every expert has rows, so that CTA 0's last unit has a stage to leave out: one unit per CTA (tiny), several units of
# fewer blocks than the ring of three stages, and of more
WGRAD = {"tiny": (64, 128, 256, 8, 2, None, "uniform"), "short": (1000, 1024, 2048, 16, 2, None, "uniform"),
         "long": (3000, 1024, 2048, 12, 2, None, "uniform"), "capacity": (1500, 1024, 2048, 12, 2, 100, "uniform")}


@pytest.mark.parametrize("op", [_gate_up_wgrad, _down_wgrad], ids=["gate_up", "down"])
@pytest.mark.parametrize("case", list(WGRAD))
def test_wait_of_a_weight_gradient_expires_and_reports(case, op):
    """CTA 0's producer never loads the first stage of its last unit, while
    the stores of the unit before may be in flight: only that unit's tile may
    be missing."""
    L = Layer(case, case=WGRAD[case])
    assert int(L.counts.min()) > 0
    L.h, L.dg, L.du, L.dy = L.rows(L.P, L.F), L.rows(L.P, L.F), L.rows(L.P, L.F), L.rows(L.P, L.H)

    def buffers():
        return [L.poison(L.E, L.F, L.H)] if op is _down_wgrad else [L.poison(L.E, L.H, L.F) for _ in range(2)]

    ref = buffers()
    op(L, L.shape, ref)
    assert L.status() == 0
    s = L.shape
    stall = moe.make_shape(s.T, s.H, s.F, s.E, s.k, C=s.C, flags=s.flags | moe.MOE_FLAG_TEST_STALL_GEMM)
    cut = buffers()
    moe.moe_set_wait_timeout_ns(50_000_000)
    try:
        op(L, stall, cut)
        status = moe.moe_read_status(L.ws, clear=True)
    finally:
        moe.moe_set_wait_timeout_ns(1_000_000_000)
    assert status == moe.MOE_DEV_GEMM_TIMEOUT, hex(status)
    missing = 0
    for a, b in zip(_bits(cut), _bits(ref)):
        missing += int((a != b).sum())
    assert 0 < missing <= 256 * 256 * 2, "bytes of the unit that was left out: %d" % missing
    got = buffers()
    op(L, s, got)
    assert L.status() == 0
    for a, b in zip(_bits(got), _bits(ref)):
        assert torch.equal(a, b)
