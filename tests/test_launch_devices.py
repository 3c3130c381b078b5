"""Every launch on every device of a process, without a GPU: the library's own
objects linked with a fake CUDA runtime (fake_cudart.cpp) that keeps each
kernel's shared-memory limit per device and refuses a launch above it, as the
runtime does."""
import ctypes
import glob
import os
import subprocess
import sys
import threading

import pytest

import grouped_expert_gemm_router_b200 as moe
from grouped_expert_gemm_router_b200 import build as moe_build

HERE = os.path.dirname(os.path.abspath(__file__))
PTR = 1 << 20  # aligned, never dereferenced: nothing runs

# entry point -> what its arguments after the shape are: p a pointer, an int itself
CALLS = {
    "moe_route": "pppppppp",
    "moe_route_dispatch": "pppppppppppp",
    "moe_grouped_swiglu": "pppppp",
    "moe_grouped_swiglu_gather": "ppppppp",
    "moe_grouped_down": "ppppp",
    "moe_grouped_down_combine": "ppppppppp",
    "moe_grouped_swiglu_fp8": "pppppppppp",  # with src_token: rows gathered
    "moe_grouped_swiglu_fp8 ": "pp0ppppppp",  # on permuted rows
    "moe_grouped_down_fp8": "ppppppp",
    "moe_grouped_down_fp8_combine": "ppppppppppp",
    "moe_grouped_swiglu_checkpoint": "ppppppppp",
    "moe_combine_backward": "ppppppppp",
    "moe_gather_backward": "pppp",
    "moe_grouped_down_backward": "pppppppppp",
    "moe_grouped_swiglu_backward": "ppppppp",
    "moe_grouped_swiglu_wgrad": "ppppppp",
    "moe_grouped_down_wgrad": "ppppp",
}
# T, H, F, E, k: the router's small and large tiles, and its tensor-core form
SHAPES = [(16, 4096, 256, 8, 2), (200, 2048, 256, 64, 4), (300, 2048, 256, 128, 8), (64, 2048, 256, 256, 8),
          (4096, 2048, 256, 128, 8)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    moe_build.build()
    objs = sorted(glob.glob(os.path.join(moe_build.HERE, "_build", "*.cu.o")))
    if len(objs) != len(moe_build.sources()):
        moe_build.build(force=True)
        objs = sorted(glob.glob(os.path.join(moe_build.HERE, "_build", "*.cu.o")))
    path = str(tmp_path_factory.mktemp("fake") / "libmoe_fake.so")
    subprocess.check_call([os.environ.get("NVCC", "nvcc"), "-cudart", "none", "-shared", "-std=c++17",
                           "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic", "-o", path,
                           os.path.join(HERE, "fake_cudart.cpp"), *objs])
    return load(path)


def load(path):
    fake, real = ctypes.CDLL(path), moe.load_library()
    for name in set(n.strip() for n in CALLS) | {"moe_forward", "moe_forward_checkpoint", "moe_backward"}:
        getattr(fake, name).argtypes = getattr(real, name).argtypes
    return fake


def _args(cls):
    a = cls()
    for n, t in cls._fields_:
        setattr(a, n, PTR if t is ctypes.c_void_p else 1)
    return a


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_entry_point_launches_on_every_device(lib, shape):
    s = moe.make_shape(*shape)
    for dev in (0, 1):
        lib.fake_set_device(dev)
        for name, form in CALLS.items():
            before = lib.fake_launches()
            st = getattr(lib, name.strip())(ctypes.byref(s), *(PTR if c == "p" else None for c in form))
            assert st == 0 and lib.fake_launches() > before, (name, "device %d" % dev, st)
        for st in (lib.moe_forward(ctypes.byref(s), ctypes.byref(_args(moe.MoeForwardArgs)), PTR, None),
                   lib.moe_forward_checkpoint(ctypes.byref(s), ctypes.byref(_args(moe.MoeForwardArgs)), PTR, PTR, PTR,
                                              PTR, None),
                   lib.moe_backward(ctypes.byref(s), ctypes.byref(_args(moe.MoeBackwardArgs)), PTR, None)):
            assert st == 0, "device %d" % dev


def test_the_fake_runtime_refuses_a_launch_above_the_limit(lib):
    """What the test above rests on: a launch of more than 48 KB fails on a
    device where the kernel's limit was not raised."""
    func = ctypes.c_char(b"f")
    cfg = (ctypes.c_uint32 * 16)()  # grid, block (3 + 3 words), dynamic shared memory (64 bits), stream, attributes
    cfg[6] = 48 * 1024 + 1
    launch, raise_limit = lib.cudaLaunchKernelExC, lib.cudaFuncSetAttribute
    lib.fake_set_device(0)
    assert raise_limit(ctypes.byref(func), 8, 64 * 1024) == 0
    assert launch(cfg, ctypes.byref(func), None) == 0
    lib.fake_set_device(1)
    assert launch(cfg, ctypes.byref(func), None) == 1
    lib.fake_set_device(0)


def first_calls_of_two_threads(path):
    """In a process of its own: the first GEMM launches of the process, two at once."""
    lib = load(path)
    s = moe.make_shape(64, 128, 256, 8, 2)
    status = []
    for name, n in (("moe_grouped_down", 5), ("moe_grouped_down_wgrad", 5)):
        lib.fake_fail_lookups(1)
        assert getattr(lib, name)(ctypes.byref(s), *[PTR] * n) != 0  # nothing found: refused, and looked up again
        before = lib.fake_lookups()
        start = threading.Barrier(2)

        def call():
            start.wait()
            status.append(getattr(lib, name)(ctypes.byref(s), *[PTR] * n))

        threads = [threading.Thread(target=call) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert lib.fake_lookups() - before == 1, "%s: %d threads looked the encoder up" % (
            name, lib.fake_lookups() - before)
    assert status == [0] * 4, status


def test_first_calls_of_two_threads_look_the_encoder_up_once(lib):
    code = "import test_launch_devices as t; t.first_calls_of_two_threads(%r)" % lib._name
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE)]))
    subprocess.run([sys.executable, "-c", code], check=True, env=env, timeout=120)
