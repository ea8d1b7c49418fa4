"""How the layer operators set up their launches, on the CPU: the library's
own objects linked with a stand-in for the CUDA runtime (tests/c/
fake_cudart.cpp), which runs no kernel but checks each launch against what its
kernel was allowed.  Calls that fail or interleave on a GPU only by chance are
made to here."""
import ctypes
import os
import shutil
import subprocess
import threading

import pytest

from collective_communication_algorithms_virtual_gb300 import build, lib

from . import test_layer_host as host
from .test_c_abi import ROOT, _cuda_home

OK, CUDA = 0, 3


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    """The library's objects and the stand-in, compiled."""
    cxx, cuda = shutil.which("g++"), os.path.join(_cuda_home(), "lib64")
    if cxx is None or not os.path.exists(os.path.join(cuda, "libcudart.so")):
        pytest.skip("no C++ compiler or no shared CUDA runtime")
    build.build()
    objs = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True)
    fake = str(tmp_path_factory.mktemp("fake") / "fake.o")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-fvisibility=hidden", "-Wall", "-Werror", "-I",
                    os.path.join(_cuda_home(), "include"), "-c", os.path.join(ROOT, "tests", "c", "fake_cudart.cpp"),
                    "-o", fake], check=True)
    return [*objs, fake], cuda


@pytest.fixture
def L(objects, tmp_path):
    """A library of its own for each test: what it keeps of kernels starts anew."""
    objs, cuda = objects
    so = str(tmp_path / "libfaked.so")
    subprocess.run([shutil.which("g++"), "-shared", "-o", so, *objs, "-L", cuda, "-lcudart", f"-Wl,-rpath,{cuda}"], check=True)
    faked, real = ctypes.CDLL(so), lib()
    for name in ("vc_reduce_scatter_norm", "vc_reduce_scatter_norm_backward", "vc_route", "vc_dispatch_plan",
                 "vc_dispatch", "vc_combine", "vc_combine_backward", "vc_last_error"):
        getattr(faked, name).argtypes = getattr(real, name).argtypes
        getattr(faked, name).restype = getattr(real, name).restype
    faked.fake_reset()
    return faked


def launches(L):
    """(grid, block, dynamic shared memory, cluster, status) of each so far."""
    out = []
    for i in range(L.fake_launches()):
        five = (ctypes.c_int * 5)()
        L.fake_launch(i, five)
        out.append(tuple(five))
    return out


SIZED = {  # kernels whose shared memory goes by the call: a larger and a smaller call
    "plan": [lambda L: host.plan(L, E=1024), lambda L: host.plan(L, E=512)],
    "norm": [lambda L: host.norm(L, H=49152), lambda L: host.norm(L, H=40001)],
    "norm to 8 bits": [lambda L: host.norm(L, H=49152, odt=host.I8), lambda L: host.norm(L, H=40001, odt=host.I8)],
    "norm backward": [lambda L: host.grad(L, rows=1, H=49152), lambda L: host.grad(L, rows=1, H=40001)],
}


@pytest.mark.parametrize("what", SIZED)
def test_first_calls_of_two_sizes_may_race(L, what):
    """A thread that has raised a kernel's shared memory is held there while
    another makes a smaller first call.  Both go through, and so does every
    later call of either size."""
    large, small = SIZED[what]
    status = {}
    L.fake_hold_next_setter()
    first = threading.Thread(target=lambda: status.update(first=large(L)))
    first.start()
    assert L.fake_wait_held()
    second = threading.Thread(target=lambda: status.update(second=small(L)))
    second.start()
    for t in (first, second):
        t.join(30)
        assert not t.is_alive()
    assert status == {"first": OK, "second": OK}, L.vc_last_error()
    assert large(L) == OK and small(L) == OK, L.vc_last_error()
    assert all(five[-1] == 0 for five in launches(L))


@pytest.mark.parametrize("largest", [16, 8])
def test_plan_takes_a_cluster_that_the_device_can_place(L, largest):
    """16 blocks where a cluster of them fits the device, else the portable 8."""
    L.fake_largest_cluster(largest)
    for rows in (2000, 40000):
        assert host.plan(L, rows=rows, topk=4, E=1024, cap=1 << 20,
                         **{k: host.ptrs(host.area(i), 2, 1 << 28) for i, k in enumerate(("ids", "slots", "offsets"))}) == OK
    assert host.plan(L, rows=4) == OK, L.vc_last_error()
    got = launches(L)
    assert [(grid, cluster) for grid, _, _, cluster, _ in got] == [(largest, largest)] * 2 + [(1, 1)]
    assert all(five[-1] == 0 for five in got)


def test_dispatch_of_no_elements_moves_scales(L):
    """Rows of no elements have nothing to move but their scales."""
    assert host.dispatch(L, H=0) == OK and launches(L) == []
    scales = dict(scale=host.ptrs(host.area(3)), recv_scale=host.ptrs(host.area(4)))
    assert host.dispatch(L, H=0, **scales) == OK
    assert [five[0] for five in launches(L)] == [1]
    assert host.dispatch(L, H=0, rows=0, **scales) == OK and len(launches(L)) == 1
