"""What the training binding hands to the library (a stand-in that records it)."""
import ctypes
import types

import pytest

import grouped_expert_gemm_router_b200 as moe

PTR = 1 << 20


@pytest.fixture
def seen(monkeypatch):
    calls = []

    def moe_backward(shape, args, ws, stream):
        calls.append({n: getattr(args._obj, n) for n, _ in moe.MoeBackwardArgs._fields_})
        return 0

    monkeypatch.setattr(moe, "load_library", lambda: types.SimpleNamespace(moe_backward=moe_backward))
    return calls


@pytest.mark.parametrize("in_args", [False, True])
@pytest.mark.parametrize("asked", [False, True])
def test_rebuild_dispatch_holds_with_prepared_args_too(seen, in_args, asked):
    """rebuild_dispatch=True is not lost when args are given; args that ask for it keep it; neither is changed."""
    s = moe.make_shape(64, 128, 256, 8, 2)
    bufs = {n: PTR + 256 * i for i, (n, _) in enumerate(moe.MoeBackwardArgs._fields_) if n != "rebuild_dispatch"}
    a = moe.backward_args(bufs, rebuild_dispatch=in_args)
    before = bytes(a)
    moe.moe_backward(s, bufs, PTR, stream=0, args=a, rebuild_dispatch=asked)
    moe.moe_backward(s, bufs, PTR, stream=0, rebuild_dispatch=asked)
    assert bytes(a) == before
    given, built = seen
    assert given.pop("rebuild_dispatch") == int(in_args or asked)
    assert built.pop("rebuild_dispatch") == int(asked)
    assert given == built == bufs
    assert ctypes.sizeof(a) == len(before)
