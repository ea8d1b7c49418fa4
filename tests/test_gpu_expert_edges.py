"""Edges of the experts' products that tests/test_gpu_expert.py does not reach,
within the same bounds."""
import time

import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import expert_ref as ref
from .layer_ref import DT, f64
from .test_gpu_expert import check, gpu, host, inputs, offsets_of  # noqa: F401

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
