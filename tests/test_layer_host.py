"""What the layer operators refuse, on the CPU: the library's own argument
checks come before any CUDA call, and the binding's tensor checks before the
library.  Buffers are made-up addresses that nothing reads."""
import ctypes
import math
import struct
import subprocess

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc
from collective_communication_algorithms_virtual_gb300 import binding as b

from .test_binding_checks import Recorder

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, I32, F16, I8 = range(5)


@pytest.fixture(scope="module")
def L():
    from collective_communication_algorithms_virtual_gb300 import build

    build.build()
    return vc.lib()


def ptrs(base, n=2, step=1 << 20):
    return (ctypes.c_void_p * n)(*[base + i * step for i in range(n)])


def area(i):
    """Addresses of argument i, far from the others'."""
    return (i + 1) << 32


def norm(L, N=2, rows=4, H=8, eps=1e-6, dt=F32, odt=F32, **over):
    a = dict(send=ptrs(area(0)), residual=ptrs(area(1)), weight=ptrs(area(2)), residual_out=ptrs(area(3)),
             out=ptrs(area(4)), scale=ptrs(area(5)), rstd=ptrs(area(6)))
    a.update(over)
    return L.vc_reduce_scatter_norm(a["send"], a["residual"], a["weight"], a["residual_out"], a["out"], a["scale"],
                                    a["rstd"], N, rows, H, eps, dt, odt, None)


@pytest.mark.parametrize("over,status", [
    (dict(N=0), INVALID), (dict(N=65), INVALID), (dict(H=49153), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(dt=I32, odt=I32), UNSUPPORTED), (dict(dt=I8, odt=I8), UNSUPPORTED), (dict(dt=9, odt=9), INVALID),
    (dict(dt=F32, odt=BF16), UNSUPPORTED), (dict(rows=1 << 31), INVALID), (dict(rows=1 << 62), INVALID),
    (dict(send=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID),
    (dict(odt=I8, scale=None), INVALID), (dict(send=ptrs(0, 2, 0)), INVALID),
    (dict(send=ptrs(area(0) + 2)), INVALID),                      # not aligned to its element
    (dict(out=ptrs(area(0))), INVALID),                           # an output over an input
    (dict(out=ptrs(area(4), 2, 64)), INVALID),                    # the ranks' outputs over each other
    (dict(residual_out=ptrs(area(1) + 16)), INVALID),             # over the residual, but not in place
    (dict(rstd=ptrs(area(4) + 32)), INVALID),
])
def test_norm_refuses(L, over, status):
    assert norm(L, **over) == status, L.vc_last_error()
    assert L.vc_last_error()


def test_empty_calls_are_accepted_without_a_gpu(L):
    assert norm(L, rows=0) == OK and norm(L, H=0) == OK
    how = b._pack_how(0, 1, 1, 1, 1, 1, 1.0)
    assert L.vc_route(ptrs(area(0)), None, ptrs(area(1)), ptrs(area(2)), 2, 0, 8, how, F32, None) == OK
    assert L.vc_combine(ptrs(area(0)), ptrs(area(1)), None, ptrs(area(2)), 2, 0, 8, 2, 4, F32, None) == OK


def grad(L, N=2, rows=4, H=8, dt=F32, **over):
    a = dict(dout=ptrs(area(0)), dro=None, h=ptrs(area(1)), weight=ptrs(area(2)), rstd=ptrs(area(3)),
             dsend=ptrs(area(4)), dres=ptrs(area(5)), dw=ptrs(area(6)))
    a.update(over)
    return L.vc_reduce_scatter_norm_backward(a["dout"], a["dro"], a["h"], a["weight"], a["rstd"], a["dsend"], a["dres"],
                                             a["dw"], N, rows, H, dt, None)


@pytest.mark.parametrize("over,status", [
    (dict(dsend=None, dres=None, dw=None), INVALID), (dict(h=None), INVALID), (dict(rstd=None), INVALID),
    (dict(H=49153), UNSUPPORTED), (dict(dt=I8), UNSUPPORTED), (dict(dsend=ptrs(area(0))), INVALID),
    (dict(dres=ptrs(area(0))), INVALID), (dict(dro=ptrs(area(7)), dres=ptrs(area(7) + 16)), INVALID),
    (dict(dw=ptrs(area(6), 2, 16)), INVALID),
])
def test_norm_backward_refuses(L, over, status):
    assert grad(L, **over) == status, L.vc_last_error()


def route(L, back=False, N=2, rows=4, E=16, dt=F32, bias=None, how=True, **over):
    h = dict(score=0, topk=2, ngroups=1, topk_groups=1, group_top=1, renormalize=1, scale=1.0)
    a = dict(logits=ptrs(area(0)), ids=ptrs(area(1)), weights=ptrs(area(2)), dlogits=ptrs(area(3)))
    a.update({k: v for k, v in over.items() if k in a})
    h.update({k: v for k, v in over.items() if k in h})
    ref = b._pack_how(*h.values()) if how else None
    if back:
        return L.vc_route_backward(a["weights"], a["logits"], a["ids"], a["dlogits"], N, rows, E, ref, dt, None)
    return L.vc_route(a["logits"], bias, a["ids"], a["weights"], N, rows, E, ref, dt, None)


@pytest.mark.parametrize("over,status", [
    (dict(how=False), INVALID), (dict(score=2), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID),
    (dict(topk=0), INVALID), (dict(topk=17), INVALID), (dict(E=64, topk=33), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(dt=I32), UNSUPPORTED), (dict(dt=7), INVALID), (dict(N=65), INVALID), (dict(rows=1 << 31), INVALID),
    (dict(ids=ptrs(area(2))), INVALID),
])
def test_route_refuses(L, over, status):
    assert route(L, **over) == status, L.vc_last_error()
    if "ids" not in over:
        assert route(L, back=True, **over) == status, L.vc_last_error()


@pytest.mark.parametrize("over", [
    dict(ngroups=3), dict(ngroups=0), dict(E=64, ngroups=64), dict(ngroups=4, topk_groups=5), dict(topk_groups=0),
    dict(group_top=0), dict(group_top=3), dict(ids=ptrs(area(0))), dict(bias=ptrs(area(1))),
])
def test_route_refuses_groups_and_overlaps(L, over):
    assert route(L, **over) == INVALID, L.vc_last_error()


def plan(L, N=2, rows=4, topk=2, E=4, cap=8, ids=ptrs(area(0)), slots=ptrs(area(1)), offsets=ptrs(area(2))):
    return L.vc_dispatch_plan(ids, slots, offsets, N, rows, topk, E, cap, None)


@pytest.mark.parametrize("over", [
    dict(E=5), dict(E=0), dict(E=1026), dict(topk=0), dict(topk=33), dict(cap=0), dict(cap=1 << 30), dict(rows=1 << 30),
    dict(N=0), dict(ids=None), dict(slots=None), dict(offsets=None), dict(slots=ptrs(area(0))), dict(offsets=ptrs(area(1) + 8)),
])
def test_plan_refuses(L, over):
    assert plan(L, **over) == INVALID, L.vc_last_error()


def dispatch(L, dt=F32, N=2, rows=4, H=8, topk=2, cap=8, **over):
    a = dict(send=ptrs(area(0)), scale=None, slots=ptrs(area(1)), recv=ptrs(area(2)), recv_scale=None)
    a.update(over)
    return L.vc_dispatch(a["send"], a["scale"], a["slots"], a["recv"], a["recv_scale"], N, rows, H, topk, cap, dt, None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=I32), UNSUPPORTED), (dict(dt=8), INVALID), (dict(scale=ptrs(area(3))), INVALID),
    (dict(recv_scale=ptrs(area(3))), INVALID), (dict(recv=ptrs(area(0))), INVALID), (dict(recv=ptrs(area(2), 2, 64)), INVALID),
    (dict(slots=None), INVALID), (dict(cap=0), INVALID), (dict(topk=40), INVALID), (dict(H=1 << 41), INVALID),
    (dict(H=1 << 39, cap=1 << 29), INVALID),
])
def test_dispatch_refuses(L, over, status):
    assert dispatch(L, **over) == status, L.vc_last_error()


def combine(L, dt=F32, N=2, rows=4, H=8, topk=2, cap=8, **over):
    a = dict(recv=ptrs(area(0)), slots=ptrs(area(1)), weights=None, out=ptrs(area(2)))
    a.update(over)
    return L.vc_combine(a["recv"], a["slots"], a["weights"], a["out"], N, rows, H, topk, cap, dt, None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=I8), UNSUPPORTED), (dict(out=None), INVALID), (dict(out=ptrs(area(0) + 64)), INVALID),
    (dict(weights=ptrs(area(2))), INVALID), (dict(N=-1), INVALID),
])
def test_combine_refuses(L, over, status):
    assert combine(L, **over) == status, L.vc_last_error()


def test_combine_backward_refuses(L):
    a = [ptrs(area(i)) for i in range(6)]
    tail = (2, 4, 8, 2, 8, F32, None)
    assert L.vc_combine_backward(a[0], a[1], a[2], None, None, None, *tail) == INVALID   # nothing asked for
    assert L.vc_combine_backward(a[0], None, a[2], None, None, a[5], *tail) == INVALID   # dweights want recv
    assert L.vc_combine_backward(a[0], a[1], a[2], None, a[1], None, *tail[:-2], I8, None) == UNSUPPORTED
    assert L.vc_combine_backward(a[0], a[1], a[2], None, a[1], a[5], *tail) == INVALID   # drecv over recv


def test_collectives_refuse_int8(L):
    p = ptrs(area(0)), ptrs(area(1))
    assert L.vc_allreduce(*p, 2, 16, I8, 0, 0, None) == INVALID


class Fake:
    """What the binding reads of a tensor, with each property settable."""

    def __init__(self, *shape, dtype=torch.float32, dev=0, contiguous=True, ptr=1 << 20):
        self.shape, self.dtype, self._dev, self._contig, self._ptr = shape, dtype, dev, contiguous, ptr
        self.device = f"cuda:{dev}" if dev >= 0 else "cpu"

    def get_device(self):
        return self._dev

    def is_contiguous(self):
        return self._contig

    def data_ptr(self):
        return self._ptr

    @property
    def nbytes(self):
        return math.prod(self.shape) * self.dtype.itemsize

    def __len__(self):
        return self.shape[0]


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(b, "lib", lambda: r)
    monkeypatch.setattr(b, "CHECK_TENSORS", True)
    return r


I = torch.int32


def test_sizes_reach_the_library(rec):
    b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(8), Fake(2, 3, 8), stream=1)
    b.vc_reduce_scatter_norm([Fake(6, 8)] * 2, [Fake(8)] * 2, Fake(2, 3, 8, dtype=torch.int8), scale=Fake(2, 3), stream=1)
    b.vc_route(Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 4), stream=1)
    b.vc_dispatch_plan(Fake(2, 3, 4, dtype=I), Fake(2, 3, 4, dtype=I), Fake(2, 9, dtype=I), 12, stream=1)
    b.vc_dispatch(Fake(2, 3, 8), Fake(2, 3, 4, dtype=I), Fake(2, 12, 8), stream=1)
    b.vc_combine(Fake(2, 12, 8), Fake(2, 3, 4, dtype=I), Fake(2, 3, 8), stream=1)
    names = [c[0] for c in rec.calls]
    assert names == ["vc_reduce_scatter_norm"] * 2 + ["vc_route", "vc_dispatch_plan", "vc_dispatch", "vc_combine"]
    args = [c[1] for c in rec.calls]
    assert args[0][7:10] == (2, 3, 8) and args[0][11:13] == (F32, F32)
    assert args[1][7:10] == (2, 3, 8) and args[1][11:13] == (F32, I8)
    assert args[2][4:7] == (2, 3, 16)
    assert args[3][3:8] == (2, 3, 4, 16, 12)
    assert args[4][5:11] == (2, 3, 8, 4, 12, F32)
    assert args[5][4:10] == (2, 3, 8, 4, 12, F32)
    # a stacked tensor's ranks lie one behind another; one weight stands for all
    assert struct.unpack("2Q", args[0][0]) == (1 << 20, (1 << 20) + 6 * 8 * 4)
    assert struct.unpack("2Q", args[0][2]) == (1 << 20, 1 << 20)


@pytest.mark.parametrize("bad", [
    lambda: b.vc_reduce_scatter_norm(Fake(2, 5, 8), Fake(8), Fake(2, 3, 8), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(9), Fake(2, 3, 8), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8, contiguous=False), Fake(8), Fake(2, 3, 8), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8, dev=-1), Fake(8), Fake(2, 3, 8), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(8), Fake(2, 3, 8, dtype=torch.int8), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(8), Fake(2, 3, 8), residual=Fake(2, 3, 8, dtype=torch.float16), stream=1),
    lambda: b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(8), Fake(2, 3, 8), rstd=Fake(2, 3, dev=1), stream=1),
    lambda: b.vc_reduce_scatter_norm([Fake(6, 8)] * 2, Fake(8), [Fake(3, 8)], stream=1),
    lambda: b.vc_route(Fake(2, 3, 16), Fake(2, 3, 4), Fake(2, 3, 4), stream=1),
    lambda: b.vc_route(Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 5), stream=1),
    lambda: b.vc_route(Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 4), bias=Fake(15), stream=1),
    lambda: b.vc_route_backward(Fake(2, 3, 4), Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 15), stream=1),
    lambda: b.vc_dispatch_plan(Fake(2, 3, 4, dtype=I), Fake(2, 3, 4, dtype=I), Fake(3, 9, dtype=I), 12, stream=1),
    lambda: b.vc_dispatch_plan(Fake(2, 3, 4, dtype=I), Fake(2, 3, 4, dtype=I), Fake(2, 9, dtype=I), 0, stream=1),
    lambda: b.vc_dispatch(Fake(2, 3, 8), Fake(2, 3, 4, dtype=I), Fake(2, 12, 9), stream=1),
    lambda: b.vc_dispatch(Fake(2, 3, 8), Fake(2, 4, 4, dtype=I), Fake(2, 12, 8), stream=1),
    lambda: b.vc_combine(Fake(2, 12, 8), Fake(2, 3, 4, dtype=I), Fake(2, 3, 8), weights=Fake(2, 3, 3), stream=1),
    lambda: b.vc_combine_backward(Fake(2, 3, 8), None, Fake(2, 3, 4, dtype=I), stream=1),
])
def test_mismatched_tensors_never_reach_the_library(rec, bad):
    with pytest.raises(b.VCError) as e:
        bad()
    assert e.value.status == b.VC_ERR_INVALID_ARG
    assert rec.calls == []


def test_header_and_checks_from_c(tmp_path):
    from .test_c_abi import _build_c_program

    out = subprocess.run([str(_build_c_program(tmp_path, "abi_layer"))], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok"), (out.returncode, out.stderr)
