"""What the experts' operators refuse, on the CPU: the library's own argument
checks come before any CUDA call, and the binding's tensor checks before the
library.  Buffers are made-up addresses that nothing reads."""
import ctypes
import struct

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc
from collective_communication_algorithms_virtual_gb300 import binding as b

from .test_binding_checks import Recorder  # noqa: F401
from .test_layer_host import BF16, F16, F32, I8, I32, INVALID, OK, UNSUPPORTED, L, area, ptrs  # noqa: F401
from .test_layer_launch_host import launches, objects  # noqa: F401
from .test_layer_launch_host import L as faked  # noqa: F401

WIDE = (1 << 20) + 1


def product(L, N=2, E=4, cap=8, win=16, width=24, tr=0, dt=BF16, **over):  # noqa: F811
    a = dict(rows=ptrs(area(0)), weight=ptrs(area(1)), offsets=ptrs(area(2)), out=ptrs(area(3)))
    a.update(over)
    return L.vc_expert_product(a["rows"], a["weight"], a["offsets"], a["out"], N, E, cap, win, width, tr, dt, None)


SIZES = [
    (dict(N=0), INVALID), (dict(N=65), INVALID), (dict(E=0), INVALID), (dict(E=3), INVALID), (dict(E=1026), INVALID),
    (dict(win=WIDE), UNSUPPORTED), (dict(width=WIDE), UNSUPPORTED), (dict(cap=1 << 31), INVALID), (dict(cap=0x7fff0001), INVALID),
    (dict(cap=1 << 62), INVALID),
    (dict(rows=None), INVALID), (dict(offsets=None), INVALID), (dict(weight=ptrs(0, 2, 0)), INVALID),
    (dict(offsets=ptrs(area(2) + 2)), INVALID),
]


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(dt=I32), UNSUPPORTED), (dict(dt=I8), UNSUPPORTED), (dict(dt=9), INVALID),
    (dict(rows=ptrs(area(0) + 1)), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID),
    (dict(out=ptrs(area(0))), INVALID), (dict(out=ptrs(area(1) + 16)), INVALID), (dict(out=ptrs(area(3), 2, 64)), INVALID),
])
def test_product_refuses(L, over, status):  # noqa: F811
    assert product(L, **over) == status, L.vc_last_error()
    assert L.vc_last_error()


def test_products_of_nothing_are_accepted_without_a_gpu(L):  # noqa: F811
    assert product(L, cap=0) == OK and product(L, width=0) == OK
    assert grad(L, win=0, width=0) == OK and grad(L, cap=0, dw=None) == OK
    assert fp8(L, cap=0) == OK and fp8(L, width=0) == OK
    assert quantize(L, rows=0) == OK and quantize(L, width=0) == OK and quantize(L, mats=0) == OK


def grad(L, N=2, E=4, cap=8, win=16, width=24, dt=BF16, wdt=None, **over):  # noqa: F811
    a = dict(dout=ptrs(area(0)), rows=ptrs(area(1)), weight=ptrs(area(2)), offsets=ptrs(area(3)), dx=ptrs(area(4)), dw=ptrs(area(5)))
    a.update(over)
    return L.vc_expert_product_backward(a["dout"], a["rows"], a["weight"], a["offsets"], a["dx"], a["dw"], N, E, cap, win,
                                        width, 1, dt, dt if wdt is None else wdt, None)


@pytest.mark.parametrize("over,status", [x for x in SIZES if "rows" not in x[0] and "offsets" not in x[0]] + [
    (dict(dx=None, dw=None), INVALID), (dict(rows=None), INVALID), (dict(dout=None), INVALID), (dict(wdt=F16), UNSUPPORTED),
    (dict(wdt=I32), UNSUPPORTED), (dict(dx=ptrs(area(0))), INVALID), (dict(dw=ptrs(area(4) + 32)), INVALID),
    (dict(wdt=F32, dw=ptrs(area(5) + 2)), INVALID),
])
def test_product_backward_refuses(L, over, status):  # noqa: F811
    assert grad(L, **over) == status, L.vc_last_error()


def fp8(L, N=2, E=4, cap=8, win=16, width=24, dt=BF16, **over):  # noqa: F811
    a = dict(rows=ptrs(area(0)), rs=ptrs(area(1)), weight=ptrs(area(2)), ws=ptrs(area(3)), offsets=ptrs(area(4)), out=ptrs(area(5)))
    a.update(over)
    return L.vc_expert_product_fp8(a["rows"], a["rs"], a["weight"], a["ws"], a["offsets"], a["out"], N, E, cap, win, width, dt, None)


@pytest.mark.parametrize("over,status", [x for x in SIZES if "offsets" not in x[0] or x[0]["offsets"] is None] + [
    (dict(dt=I8), UNSUPPORTED), (dict(rs=None), INVALID), (dict(ws=ptrs(area(3) + 2)), INVALID), (dict(out=ptrs(area(1))), INVALID),
    (dict(out=ptrs(area(5) + 1)), INVALID),
])
def test_product_fp8_refuses(L, over, status):  # noqa: F811
    assert fp8(L, **over) == status, L.vc_last_error()


def quantize(L, N=2, mats=1, rows=8, width=40, block=1, dt=BF16, count=None, **over):  # noqa: F811
    a = dict(x=ptrs(area(0)), out=ptrs(area(1)), scale=ptrs(area(2)))
    a.update(over)
    return L.vc_quantize_fp8(a["x"], a["out"], a["scale"], count, N, mats, rows, width, block, dt, None)


@pytest.mark.parametrize("over,status", [
    (dict(N=0), INVALID), (dict(block=2), UNSUPPORTED), (dict(block=0), UNSUPPORTED), (dict(dt=I8), UNSUPPORTED), (dict(dt=7), INVALID),
    (dict(width=WIDE), UNSUPPORTED), (dict(rows=1 << 31), INVALID), (dict(mats=1 << 20, rows=1 << 20), INVALID),
    (dict(count=ptrs(area(3)), block=128), INVALID), (dict(count=ptrs(area(3)), mats=2), INVALID),
    (dict(count=ptrs(area(3) + 1)), INVALID), (dict(x=None), INVALID), (dict(scale=None), INVALID), (dict(out=ptrs(area(0))), INVALID),
    (dict(scale=ptrs(area(1) + 16)), INVALID), (dict(x=ptrs(area(0) + 1)), INVALID),
])
def test_quantize_refuses(L, over, status):  # noqa: F811
    assert quantize(L, **over) == status, L.vc_last_error()


def clip(L, grads, counts, dtypes, N=1, out=None, norm=None, max_norm=1.0, across=1):  # noqa: F811
    n = len(grads)
    at = struct.pack(f"={n}Q", *grads)
    return L.vc_clip_grad_norm(at, at if out == "in place" else None if out is None else struct.pack(f"={n}Q", *out),
                               struct.pack(f"={n}Q", *counts), struct.pack(f"={len(dtypes)}i", *dtypes), N, len(dtypes),
                               norm if norm is not None else ptrs(area(9), N, 64), max_norm, across, None)


A = area(0)


@pytest.mark.parametrize("args,status", [
    (dict(grads=[A], counts=[4], dtypes=[I32]), UNSUPPORTED), (dict(grads=[A], counts=[4], dtypes=[9]), INVALID),
    (dict(grads=[0], counts=[4], dtypes=[F32]), INVALID), (dict(grads=[A + 2], counts=[4], dtypes=[F32]), INVALID),
    (dict(grads=[A + 1], counts=[4], dtypes=[BF16]), INVALID), (dict(grads=[A], counts=[1 << 41], dtypes=[BF16]), INVALID),
    (dict(grads=[A, A], counts=[1 << 40, 1 << 40], dtypes=[F32, F32]), INVALID), (dict(grads=[A], counts=[4], dtypes=[F32], N=0), INVALID),
    (dict(grads=[A], counts=[4], dtypes=[F32], out="in place", max_norm=-1.0), INVALID),
    (dict(grads=[A], counts=[4], dtypes=[F32], out="in place", max_norm=float("nan")), INVALID),
    (dict(grads=[A, A + 8], counts=[4, 4], dtypes=[F32, F32], out="in place"), INVALID),   # one gradient over another
    (dict(grads=[A], counts=[4], dtypes=[F32], out=[A + 8]), INVALID),                     # an output over its gradient
    (dict(grads=[A, A + 64], counts=[4, 4], dtypes=[F32, F32], out=[A + 64, A + 128]), INVALID),  # over another's
    (dict(grads=[A], counts=[16], dtypes=[F32], norm=ptrs(A + 8, 1)), INVALID),            # the norm over a gradient
    (dict(grads=[A], counts=[16], dtypes=[F32], norm=ptrs(area(9) + 2, 1)), INVALID),
    (dict(grads=[A, A + 64], counts=[4, 4], dtypes=[F32], N=2, norm=ptrs(area(9), 2, 0)), INVALID),
])
def test_clip_refuses(L, args, status):  # noqa: F811
    assert clip(L, **args) == status, L.vc_last_error()


def test_no_array_is_refused(L):  # noqa: F811
    assert L.vc_clip_grad_norm(None, None, None, None, 1, 1, ptrs(A, 1), 1.0, 1, None) == INVALID
    assert L.vc_clip_grad_norm(None, None, None, None, 1, 0, None, 1.0, 1, None) == INVALID


class TestLaunches:
    """How the calls are launched, against a stand-in for the CUDA runtime."""

    @pytest.fixture
    def F(self, faked):  # noqa: F811
        real = vc.lib()
        for name in ("vc_quantize_fp8", "vc_clip_grad_norm", "vc_expert_product"):
            getattr(faked, name).argtypes, getattr(faked, name).restype = getattr(real, name).argtypes, getattr(real, name).restype
        return faked

    def test_clip_takes_a_launch_for_each_pass_and_table(self, F):
        step = 1 << 20
        for tensors, N, tables in ((1, 1, 1), (96, 1, 1), (97, 1, 1), (768, 1, 1), (769, 1, 2), (400, 4, 3)):
            F.fake_reset()
            n = tensors * N
            args = dict(grads=[A + i * step for i in range(n)], counts=[1000] * n, dtypes=[BF16] * tensors, N=N,
                        norm=ptrs(A - (1 << 20), N, 64))
            assert clip(F, out="in place", **args) == OK, F.vc_last_error()
            assert len(launches(F)) == 2 * tables
            F.fake_reset()
            assert clip(F, **args) == OK and len(launches(F)) == tables + 1
            assert all(five[-1] == 0 for five in launches(F))

    def test_clip_of_runs_that_interleave(self, F):
        """Tensors of two ranks in turn in one buffer, in any order, are apart."""
        at = [A + i * 4096 for i in (0, 2, 4, 5, 3, 1)]
        assert clip(F, grads=at, counts=[100] * 6, dtypes=[F32] * 3, N=2, out="in place") == OK, F.vc_last_error()
        at[3] = A + 4096 * 4 + 396
        assert clip(F, grads=at, counts=[100] * 6, dtypes=[F32] * 3, N=2, out="in place") == INVALID

    def test_quantize(self, F):
        assert quantize(F, rows=100000, width=4096, x=ptrs(area(0), 2, 1 << 30), out=ptrs(area(1), 2, 1 << 30), scale=ptrs(area(2), 2, 1 << 30)) == OK
        assert quantize(F, rows=1, width=1) == OK and quantize(F, mats=3, rows=300, width=300, block=128) == OK
        assert [five[-1] for five in launches(F)] == [0, 0, 0]

    def test_fp32_products(self, F):
        assert product(F, dt=F32) == OK and product(F, dt=F32, win=0) == OK, F.vc_last_error()
        assert all(five[-1] == 0 for five in launches(F)) and len(launches(F)) == 2


# -- the binding -------------------------------------------------------------------
def test_tensors_on_the_host_are_refused():
    z, i = torch.zeros(2, 4, 8), torch.zeros(2, 3, dtype=torch.int32)
    f8 = torch.zeros(2, 4, 8, dtype=torch.float8_e4m3fn)
    s = torch.zeros(2, 4, 1)
    for call in (lambda: vc.vc_expert_product(z, torch.zeros(2, 2, 8, 8), i, z.clone()),
                 lambda: vc.vc_expert_product_backward(z, z, torch.zeros(2, 2, 8, 8), i, drows=z.clone()),
                 lambda: vc.vc_quantize_fp8(z, f8, s),
                 lambda: vc.vc_expert_product_fp8(f8, s, f8, s, i, z),
                 lambda: vc.vc_clip_grad_norm([[z]], torch.zeros(1))):
        with pytest.raises(vc.VCError) as e:
            call()
        assert e.value.status == INVALID


class Fake(torch.Tensor):
    """A host tensor that says it is on cuda:0."""

    def get_device(self):
        return 0


def on0(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


@pytest.fixture
def recorded(monkeypatch):
    calls = []

    class Rec:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0
    monkeypatch.setattr(b, "lib", lambda: Rec())
    monkeypatch.setattr(b, "_stream_handle", lambda stream, like: 7)
    return calls


def test_binding_checks_shapes_and_types(recorded):
    x, w, off, out = on0(2, 4, 8), on0(2, 3, 8, 6), on0(2, 4, dtype=torch.int32), on0(2, 4, 6)
    vc.vc_expert_product(x, w, off, out)
    name, a = recorded[-1]
    assert name == "vc_expert_product" and a[4:] == (2, 6, 4, 8, 6, False, F32, 7)
    vc.vc_expert_product(x, on0(2, 3, 6, 8), off, out, transposed=True)
    for bad in (dict(weight=on0(2, 3, 6, 8)), dict(offsets=on0(2, 4)), dict(offsets=on0(2, 1, dtype=torch.int32)), dict(out=on0(2, 5, 6)),
                dict(out=on0(2, 4, 6, dtype=torch.bfloat16)), dict(rows=on0(4, 2, 8).transpose(0, 1))):
        with pytest.raises(vc.VCError):
            vc.vc_expert_product(**{**dict(rows=x, weight=w, offsets=off, out=out), **bad})
    vc.vc_expert_product_backward(out, x, w, off, drows=on0(2, 4, 8), dweight=on0(2, 3, 8, 6))
    assert recorded[-1][1][6:] == (2, 6, 4, 8, 6, False, F32, F32, 7)
    for bad in (dict(), dict(dweight=on0(2, 3, 6, 8)), dict(rows=None, dweight=on0(2, 3, 8, 6)), dict(rows=None, drows=None, dweight=on0(2, 3, 8, 6))):
        with pytest.raises(vc.VCError):
            vc.vc_expert_product_backward(**{**dict(dout=out, rows=x, weight=w, offsets=off), **bad})


def test_binding_checks_8_bits(recorded):
    f8 = torch.float8_e4m3fn
    x = on0(2, 4, 130, dtype=torch.bfloat16)
    vc.vc_quantize_fp8(x, on0(2, 4, 130, dtype=f8), on0(2, 4, 2), offsets=on0(2, 4, dtype=torch.int32))
    a = recorded[-1][1]
    assert a[4:] == (2, 1, 4, 130, 1, BF16, 7) and struct.unpack("=2Q", a[3])[1] - struct.unpack("=2Q", a[3])[0] == 16
    vc.vc_quantize_fp8(on0(2, 3, 140, 130), on0(2, 3, 140, 130, dtype=f8), on0(2, 3, 2, 2), block_rows=128)
    assert recorded[-1][1][4:] == (2, 3, 140, 130, 128, F32, 7)
    for bad in (dict(scale=on0(2, 4, 1)), dict(out=on0(2, 4, 130, dtype=torch.int8)), dict(block_rows=64), dict(x=on0(4, 130))):
        with pytest.raises(vc.VCError):
            vc.vc_quantize_fp8(**{**dict(x=x, out=on0(2, 4, 130, dtype=f8), scale=on0(2, 4, 2)), **bad})
    good = dict(rows=on0(2, 4, 130, dtype=f8), row_scale=on0(2, 4, 2), weight=on0(2, 3, 200, 130, dtype=f8), weight_scale=on0(2, 3, 2, 2),
                offsets=on0(2, 4, dtype=torch.int32), out=on0(2, 4, 200, dtype=torch.float16))
    vc.vc_expert_product_fp8(**good)
    assert recorded[-1][1][6:] == (2, 6, 4, 130, 200, F16, 7)
    for bad in (dict(row_scale=on0(2, 4, 1)), dict(weight_scale=on0(2, 3, 2, 1)), dict(weight=on0(2, 3, 130, 200, dtype=f8)), dict(rows=on0(2, 4, 130))):
        with pytest.raises(vc.VCError):
            vc.vc_expert_product_fp8(**{**good, **bad})
    vc.vc_dispatch(on0(2, 4, 130, dtype=f8), on0(2, 4, 2, dtype=torch.int32), on0(2, 9, 130, dtype=f8))
    assert recorded[-1][0] == "vc_dispatch" and recorded[-1][1][-2] == I8


def test_binding_checks_gradients(recorded):
    grads = [[on0(5), on0(3, dtype=torch.bfloat16)], [on0(4), on0(0, dtype=torch.bfloat16)]]
    vc.vc_clip_grad_norm(grads, on0(2), max_norm=2.0, across=False)
    name, a = recorded[-1]
    assert a[0] == a[1] and struct.unpack("=4Q", a[2]) == (5, 3, 4, 0) and struct.unpack("=2i", a[3]) == (F32, BF16)
    assert a[4:6] == (2, 2) and a[7:] == (2.0, False, 7)
    vc.vc_clip_grad_norm(grads, on0(2))
    assert recorded[-1][1][1] is None
    for bad in (dict(grads=[grads[0], grads[1][:1]]), dict(grads=[grads[0], grads[1][::-1]]), dict(norm=on0(3)), dict(norm=on0(2, dtype=torch.float64)),
                dict(out=grads[:1]), dict(out=[grads[1], grads[0]]), dict(out=grads, max_norm=None), dict(grads=[[on0(6)[::2]], [on0(3)]]), dict(grads=[])):
        with pytest.raises(vc.VCError):
            vc.vc_clip_grad_norm(**{**dict(grads=grads, norm=on0(2), max_norm=1.0), **bad})
