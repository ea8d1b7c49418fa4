"""The gradients' norm at the ends of fp32's range, within the bounds of
tests/test_gpu_clip.py: they do not depend on the size of the numbers."""
import math

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .layer_ref import DT
from .test_gpu_clip import check, gpu, gradients, norms  # noqa: F401

pytestmark = pytest.mark.gpu


def clipped(grads, across=True):
    """To half of their norm, into other tensors and in place."""
    N, kept = len(grads), [[t.clone() for t in ts] for ts in grads]
    half = max(norms(kept, across)) / 2
    out, norm = [[torch.empty_like(t) for t in ts] for ts in grads], torch.full((N,), 7.0, device="cuda")
    vc.vc_clip_grad_norm(grads, norm, max_norm=half, out=out, across=across)
    check(grads, kept, norm, out, half, across)
    vc.vc_clip_grad_norm(grads, norm, max_norm=half, across=across)
    check(grads, kept, norm, grads, half, across)


# 64 squares of 2.4e18 pass fp32's largest number, one of 1.9e19 does; those of
# 1e-19 are among the subnormal ones, those of 1e-23 below them all
@pytest.mark.parametrize("size", [3e18, 2e19, 1e30, 1e36, 1e-14, 1e-20, 1e-23, 1e-25, 1e-37])
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_numbers_of_one_size(size, gap, dt):
    for sizes in ([64, 3], [40000, 1]):
        for across in (True, False):
            grads = gradients(sizes, [dt, dt], 2, gap=gap)
            for ts in grads:
                for t in ts:
                    t.copy_(torch.full_like(t, size))
            clipped(grads, across)


@pytest.mark.parametrize("size", [1e18, 1e19, 1e35, 1e-15, 1e-20, 1e-35])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_numbers_about_one_size(size, dt):
    clipped(gradients([100001, 77, 4096], [dt] * 3, 3, by=size))


@pytest.mark.parametrize("dt,least", [("f32", 2.0 ** -149), ("bf16", 2.0 ** -133)])
def test_the_smallest_numbers(dt, least):
    grads = gradients([1000, 40001], [dt, dt], 1)
    for t in grads[0]:
        t.copy_(torch.full_like(t, 4 * least))
    clipped(grads)


@pytest.mark.parametrize("one", [1e30, 1e20, 1.0, 1e-16, 1e-30])
@pytest.mark.parametrize("rest", [1e-38, 1e-25, 1e-10])
def test_one_number_among_others(one, rest):
    """In its thread's 64 and next to them; zeros around."""
    for at in (0, 3, 2049, 39999):
        grads = gradients([40000, 5000], ["f32", "bf16"], 1)
        for t in grads[0]:
            t.copy_(torch.full_like(t, rest))
        grads[0][0][at], grads[0][0][8000:9000] = one, 0
        clipped(grads)


def test_a_norm_above_fp32_is_infinite():
    for n, size, infinite in ((1, 3.4e38, False), (5, 3e38, True), (40000, 1e38, True)):
        grads = [[torch.full((n,), size, device="cuda")]]
        norm, out = torch.empty(1, device="cuda"), [[torch.empty(n, device="cuda")]]
        vc.vc_clip_grad_norm(grads, norm, max_norm=1e30, out=out)
        assert bool(torch.isinf(norm[0])) == infinite and (not infinite or bool((out[0][0] == 0).all()))


def test_infinity_and_nan_among_small_numbers():
    for bad in (math.inf, -math.inf, math.nan):
        for dt in ("f32", "bf16", "f16"):
            t = torch.full((5000,), 1e-7, dtype=DT[dt], device="cuda")
            t[1234] = bad
            norm = torch.empty(1, device="cuda")
            vc.vc_clip_grad_norm([[t]], norm)
            assert math.isnan(norm[0]) if math.isnan(bad) else norm[0] == math.inf


@pytest.mark.parametrize("across", [True, False])
@pytest.mark.parametrize("N,T", [(1, 5000), (64, 100), (3, 2500)])
def test_many_tables(N, T, across):
    """Tables of some hundred tensors each, one launch's blocks after another's
    adding to the same parts."""
    grads = gradients([1 + i % 41 + 3 * N for i in range(T)], ["bf16" if i % 5 else "f32" for i in range(T)], N)
    clipped(grads, across)
    first, again = (torch.empty(N, device="cuda") for _ in range(2))
    for norm in (first, again):
        vc.vc_clip_grad_norm(grads, norm, across=across)
    assert torch.equal(first, again)


def test_parts_do_not_grow_with_the_tables():
    """What each block of each launch adds up for the norm: as many bytes for
    eight tables of the largest tensors as for one."""
    read = []
    for T in (700, 6000):
        grads = [[torch.ones(40, device="cuda")] * T for _ in range(2)]  # the norm alone: one tensor may stand for many
        norm = torch.empty(2, device="cuda")
        vc.vc_trace_enable(True)
        vc.vc_clip_grad_norm(grads, norm)
        records = vc.vc_trace_read()
        vc.vc_trace_enable(False)
        read.append(records[-1]["bytes"])
        assert [r["step"] for r in records] == list(range(len(records))) and abs(float(norm[0]) - (80 * T) ** 0.5) < 1e-3
    assert read[0] == read[1] > 0
