"""Edges of the experts' products that tests/test_gpu_expert.py does not reach,
within the same bounds."""
import time

import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import expert_ref as ref
from .layer_ref import DT, f64
from .test_gpu_expert import check, gpu, host, inputs  # noqa: F401
from .test_gpu_fp8 import blocks, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("wide", [False, True])
def test_the_rows_behind_an_expert_are_nan(dt, wide):
    """The last step of a sum over ragged rows loads the next expert's, which
    both blocks of a pair set to 0 before the products read them: every other
    expert's rows are NaN here, on both sides, and no other gradient is."""
    rows = np.array([[1 + 7 * i % 79 for i in range(24)], [64 + 5 * i % 17 for i in range(24)]])
    cap, win, width = int(rows.sum(1).max()) + 40, 296, 520
    x, w, dy, off = inputs(dt, rows, cap, win, width, False)
    for d, ends in enumerate(off.tolist()):
        for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if i % 2:
                x[d][lo:hi], dy[d][lo:hi] = float("nan"), float("nan")
        x[d][ends[-1]:], dy[d][ends[-1]:] = float("inf"), float("nan")
    dw = [torch.zeros(t.shape, dtype=torch.float32 if wide else t.dtype, device="cuda") for t in w]
    vc.vc_expert_product_backward(dy, x, w, off, dweight=dw)
    X, dY = (np.nan_to_num(host(t), nan=0, posinf=0) for t in (x, dy))
    want, bound = ref.weight_grad(dY, X, off.cpu(), host(w).shape, False, "f32" if wide else dt)
    check(host(dw)[:, ::2], want[:, ::2], bound[:, ::2], "dweight")
    assert all(bool(torch.isnan(t[1::2]).all()) for t in dw)
    first = [t.clone() for t in dw]
    for _ in range(100):
        vc.vc_expert_product_backward(dy, x, w, off, dweight=dw)
        assert all(torch.equal(a[::2], b[::2]) for a, b in zip(first, dw))
    assert vc.vc_device_errors() == 0


def test_a_wait_that_runs_out_ends_the_others_and_is_reported():
    """The way out of the products' waits, in a launch with nothing in flight.
    The wait that is ended would run out by itself after some 0.3 s."""
    assert vc.vc_device_errors() == 0
    assert vc.vc_product_selftest() == 4  # the first launch loads the kernel
    begin = time.perf_counter()
    assert vc.vc_product_selftest() == 4
    assert time.perf_counter() - begin < 0.1
    side = torch.cuda.Stream()
    assert vc.vc_product_selftest(side) == 4 and vc.vc_device_errors() == 0
    x, w, _, off = inputs("bf16", [[40, 30]], 80, 72, 64, False)
    out = torch.zeros(1, 80, 64, dtype=DT["bf16"], device="cuda")
    vc.vc_expert_product(x, w, off, out)
    X, W = host(x), host(w)
    check(f64(out), *ref.product(X, W, off.cpu(), np.zeros(out.shape), False, "bf16"), "out")
    assert vc.vc_device_errors() == 0


OUTSIDE = [[[-5, 4, 400]], [[3, 2, 6]], [[0, 300, 300]], [[2 ** 31 - 1, -2 ** 31, 5]], [[60, -1, 70]], [[9, 9, 2]]]


@pytest.mark.parametrize("ends", OUTSIDE)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("win,width", [(64, 72), (61, 67)])
def test_offsets_outside_the_buffer_all_outputs(dt, ends, win, width):
    """Taken into [0, capacity]; an end before its beginning is an expert of no
    rows, so that no row has two.  Widths off 16-byte boundaries are copied by
    the same offsets."""
    x, w, dy, _ = inputs(dt, [[4, 4]], 70, win, width, True)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out, dx = (torch.full((1, 70, n), 7.0, dtype=DT[dt], device="cuda") for n in (width, win))
    dw = torch.full((1, 2, width, win), float("nan"), dtype=DT[dt], device="cuda")
    vc.vc_expert_product(x, w, off, out, transposed=True)
    vc.vc_expert_product_backward(dy, x, w, off, drows=dx, dweight=dw, transposed=True)
    X, W, dY = (host(t) for t in (x, w, dy))
    check(f64(out), *ref.product(X, W, off.cpu(), np.full(out.shape, 7.0), True, dt), "out")
    check(f64(dx), *ref.product(dY, W, off.cpu(), np.full(dx.shape, 7.0), False, dt), "drows")
    check(f64(dw), *ref.weight_grad(dY, X, off.cpu(), W.shape, True, dt), "dweight")


def rounded(x, B):
    """x (.., rows, width) in 8 bits by the library."""
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(*x.shape[:-2], -(-x.shape[-2] // B), blocks(x.shape[-1]), device="cuda")
    vc.vc_quantize_fp8(x, q, s, block_rows=B)
    return q, s


@pytest.mark.parametrize("ends", OUTSIDE)
@pytest.mark.parametrize("win,width", [(256, 144), (130, 67)])
def test_8_bit_offsets_outside_the_buffer(ends, win, width):
    g = torch.Generator(device="cuda").manual_seed(0)
    x8, xs = rounded(torch.randn(1, 70, win, generator=g, device="cuda"), 1)
    w8, ws = rounded(torch.randn(1, 2, width, win, generator=g, device="cuda"), 128)
    off, out = torch.tensor(ends, dtype=torch.int32, device="cuda"), torch.full((1, 70, width), 7.0, device="cuda")
    vc.vc_expert_product_fp8(x8, xs, w8, ws, off, out)
    X, W = values(x8, xs, 1), values(w8, ws, 128)
    want, bound = ref.product(X, W, off.cpu(), np.full(out.shape, 7.0), True, "f32")
    size, _ = ref.product(np.abs(X), np.abs(W), off.cpu(), np.zeros(out.shape), True, "f32")
    # a block's scale is rounded once, its sums are added by one rounding each
    check(f64(out), want, bound + (2 * blocks(win) + 1) * ref.ULP * size, "out")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_8_bit_products_over_nothing(dt):
    """in_width 0: the experts' rows are 0, the others stay."""
    f8 = torch.float8_e4m3fn
    x8, w8 = torch.empty(2, 200, 0, dtype=f8, device="cuda"), torch.empty(2, 2, 264, 0, dtype=f8, device="cuda")
    xs, ws = torch.empty(2, 200, 0, device="cuda"), torch.empty(2, 2, 3, 0, device="cuda")
    off = torch.tensor([[0, 3, 150], [7, 7, 8]], dtype=torch.int32, device="cuda")
    out = torch.full((2, 200, 264), 7.0, dtype=DT[dt], device="cuda")
    vc.vc_expert_product_fp8(x8, xs, w8, ws, off, out)
    assert bool((out[0, :150] == 0).all()) and bool((out[0, 150:] == 7).all())
    assert bool((out[1, 7] == 0).all()) and bool((out[1, :7] == 7).all()) and bool((out[1, 8:] == 7).all())
    assert vc.vc_device_errors() == 0
