"""The training entry points on the host: every refusal happens before any
CUDA call (no device is needed), the argument struct mirrors the header, and
the host view of the 8-bit checkpoint follows the documented byte order."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import grouped_expert_gemm_router_b200 as moe
from grouped_expert_gemm_router_b200 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
PTR = 1 << 20  # aligned, never dereferenced: every call below is refused on the host

# entry point -> its pointer arguments in order, with their alignment (0: may be NULL)
STEPS = {
    "moe_dispatch": [("topk_idx", 4), ("expert_counts", 4), ("expert_offsets", 4), ("src_token", 4), ("dest_row", 4)],
    "moe_grouped_swiglu_checkpoint": [("x_perm", 16), ("w_gate", 16), ("w_up", 16), ("h", 16), ("g_q", 16),
                                      ("u_q", 16), ("scale", 2)],
    "moe_combine_backward": [("dout", 16), ("y", 16), ("dest_row", 4), ("topk_w", 4), ("topk_idx", 4), ("dy", 16),
                             ("dtopk_w", 4), ("dlogits", 0)],
    "moe_grouped_down_backward": [("dy", 16), ("w_down", 16), ("g_q", 16), ("u_q", 16), ("scale", 2), ("dg", 16),
                                  ("du", 16), ("h", 16)],
    "moe_grouped_swiglu_backward": [("dg", 16), ("du", 16), ("w_gate", 16), ("w_up", 16), ("dx_perm", 16)],
    "moe_gather_backward": [("dx_perm", 16), ("dest_row", 4), ("dx", 16)],
    "moe_grouped_swiglu_wgrad": [("x_perm", 16), ("dg", 16), ("du", 16), ("dw_gate", 16), ("dw_up", 16)],
    "moe_grouped_down_wgrad": [("h", 16), ("dy", 16), ("dw_down", 16)],
}
NO_WORKSPACE = ("moe_combine_backward", "moe_gather_backward")


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load_library()


def _call(lib, name, shape, ptrs, ws=PTR):
    tail = [None] if name in NO_WORKSPACE else [ws, None]
    return getattr(lib, name)(ctypes.byref(shape), *ptrs, *tail)


@pytest.mark.parametrize("name", list(STEPS))
def test_steps_refuse_bad_pointers(lib, name):
    s = moe.make_shape(64, 128, 256, 8, 2)
    args = STEPS[name]
    for i, (what, align) in enumerate(args):
        for bad in ([None] if align else []) + ([PTR + align // 2] if align else [PTR + 2]):
            ptrs = [PTR] * len(args)
            ptrs[i] = bad
            assert _call(lib, name, s, ptrs) == INVALID, (what, bad)
    if name not in NO_WORKSPACE:
        for ws in (None, PTR + 16):
            assert _call(lib, name, s, [PTR] * len(args), ws) == WORKSPACE


@pytest.mark.parametrize("name", list(STEPS))
@pytest.mark.parametrize("bad", [dict(T=0), dict(H=96), dict(F=100), dict(E=257), dict(k=9), dict(C=-1)])
def test_steps_refuse_unsupported_shapes(lib, name, bad):
    d = dict(T=64, H=128, F=256, E=8, k=2, C=0)
    d.update(bad)
    assert _call(lib, name, moe.make_shape(**d), [PTR] * len(STEPS[name])) == UNSUPPORTED


def _backward_args(**kw):
    a = moe.MoeBackwardArgs()
    for n, _ in moe.MoeBackwardArgs._fields_:
        setattr(a, n, 1 if n == "rebuild_dispatch" else PTR)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def test_backward_refuses_before_the_first_step(lib):
    s = moe.make_shape(64, 128, 256, 8, 2)
    fields = [n for n, _ in moe.MoeBackwardArgs._fields_ if n != "rebuild_dispatch"]
    optional = {"dx", "dlogits", "dw_down"}  # NULL: not wanted
    for n in fields:
        bad = [PTR + 1] + ([] if n in optional else [None])
        for v in bad:
            assert lib.moe_backward(ctypes.byref(s), ctypes.byref(_backward_args(**{n: v})), PTR, None) == INVALID, n
    assert lib.moe_backward(ctypes.byref(s), None, PTR, None) == INVALID
    assert lib.moe_backward(ctypes.byref(s), ctypes.byref(_backward_args()), PTR + 16, None) == WORKSPACE
    bad_shape = moe.make_shape(64, 128, 100, 8, 2)
    assert lib.moe_backward(ctypes.byref(bad_shape), ctypes.byref(_backward_args()), PTR, None) == UNSUPPORTED


def test_forward_checkpoint_refuses_before_the_first_step(lib):
    s = moe.make_shape(64, 128, 256, 8, 2)

    def call(ck=(PTR, PTR, PTR), **kw):
        a = moe.MoeForwardArgs()
        for n, _ in moe.MoeForwardArgs._fields_:
            setattr(a, n, PTR)
        for n, v in kw.items():
            setattr(a, n, v)
        return lib.moe_forward_checkpoint(ctypes.byref(s), ctypes.byref(a), *ck, PTR, None)

    for n in ("x", "x_perm", "w_gate", "w_up", "w_down", "h", "y", "out"):
        assert call(**{n: None}) == INVALID and call(**{n: PTR + 8}) == INVALID, n
    for n in ("topk_idx", "topk_w", "expert_counts", "expert_offsets", "src_token", "dest_row"):
        assert call(**{n: None}) == INVALID and call(**{n: PTR + 2}) == INVALID, n
    for i in range(3):
        ck = [PTR] * 3
        ck[i] = None
        assert call(ck=ck) == INVALID
    assert lib.moe_forward_checkpoint(ctypes.byref(s), None, PTR, PTR, PTR, PTR, None) == INVALID


def test_backward_args_mirror_the_header():
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    end = text.index("} moe_backward_args;")
    body = text[text.rindex("typedef struct {", 0, end):end]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)[len("typedef struct {"):]
    names = []
    for decl in body.split(";"):
        names += re.findall(r"(\w+)\s*(?:,|$)", decl.strip())
    assert names == [n for n, _ in moe.MoeBackwardArgs._fields_]


def test_checkpoint_values_follow_the_byte_order():
    """Feature f of a block of 32 sits at byte 4 (f % 8) + f / 8, its scale is
    2^(byte - 127)."""
    P, F = 3, 96
    rng = np.random.default_rng(0)
    plain = rng.integers(0, 127, (P, F)).astype(np.uint8)  # finite codes
    scale = rng.integers(100, 150, (P, F // 32, 2)).astype(np.uint8)
    codes = np.zeros((P, F), np.uint8)
    for f in range(F):
        codes[:, f // 32 * 32 + 4 * (f % 8) + f % 32 // 8] = plain[:, f]
    for which in (0, 1):
        got = moe.checkpoint_values(torch.from_numpy(codes), torch.from_numpy(scale), which).numpy()
        want = torch.from_numpy(plain).view(torch.float8_e4m3fn).double().numpy()
        want = want * 2.0 ** (np.repeat(scale[:, :, which], 32, axis=1).astype(np.float64) - 127)
        assert np.array_equal(got.astype(np.float64), want)
