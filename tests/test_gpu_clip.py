"""The gradients' norm and clipping against 64 bits.

Squares and sums of 64 of them are fp32, so the sum of squares is within 66 u of
exact (u = 2^-24; every term is positive), its root and the store within half of
that and 2 u; the factor adds a rounding, the product another, the store its
own."""
import math

import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .layer_ref import DT, U32, f64, store_bound

pytestmark = pytest.mark.gpu
NORM = 36 * U32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gradients(sizes, types, N, seed=0, gap=0, by=1.0):
    """Each rank's tensors, one behind another in a buffer of each type, `gap`
    elements between them; of sizes[i] - rank elements where that is more than 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for r in range(N):
        mine = []
        for n, dt in zip(sizes, types):
            n = max(n - r, 0)
            room = torch.full((gap + n + 40,), 7.0, dtype=DT[dt], device="cuda")
            room[gap:gap + n] = (torch.randn(n, generator=g, device="cuda") * by).to(DT[dt])
            mine.append(room[gap:gap + n])
        out.append(mine)
    return out


def norms(grads, across):
    squares = [sum(float((f64(t) ** 2).sum()) for t in ts) for ts in grads]
    return [math.sqrt(sum(squares) if across else s) for s in squares]


def check(grads, kept, norm, out, max_norm, across):
    want = norms(kept, across)
    for r, ts in enumerate(kept):
        got = float(norm[r])
        assert abs(got - want[r]) <= NORM * want[r] + 1e-45, (got, want[r])
        limit = float(np.float32(max_norm))
        for t, o in zip(ts, out[r]):
            if got <= limit:
                assert torch.equal(o, t)
                continue
            exact = f64(t) * (limit / want[r])
            dt = {v: k for k, v in DT.items()}[t.dtype]
            bound = (NORM + 3 * U32) * np.abs(exact) + store_bound(exact, dt)
            assert (np.abs(f64(o) - exact) <= bound).all()


MIXED = ([70000, 1, 0, 513, 8, 100001, 4096], ["bf16", "f32", "bf16", "f16", "f32", "f32", "f16"])


@pytest.mark.parametrize("across", [True, False])
@pytest.mark.parametrize("gap", [0, 1, 8])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0, math.inf])
@pytest.mark.parametrize("N", [1, 3])
def test_clip(across, gap, max_norm, N):
    grads = gradients(*MIXED, N, gap=gap)
    kept = [[t.clone() for t in ts] for ts in grads]
    norm = torch.full((N,), 7.0, device="cuda")
    out = gradients(*MIXED, N, seed=1, gap=0)
    vc.vc_clip_grad_norm(grads, norm, max_norm=max_norm, out=out, across=across)
    check(grads, kept, norm, out, max_norm, across)
    assert all(torch.equal(a, b) for ts, ks in zip(grads, kept) for a, b in zip(ts, ks))
    vc.vc_clip_grad_norm(grads, norm, max_norm=max_norm, across=across)  # in place
    check(grads, kept, norm, grads, max_norm, across)
    again = torch.empty_like(norm)
    vc.vc_clip_grad_norm(kept, again, across=across)
    assert torch.equal(again, norm)


def test_elements_around_the_tensors_stay():
    for N, gap in ((2, 3), (1, 8)):
        grads = gradients(*MIXED, N, gap=gap)
        vc.vc_clip_grad_norm(grads, torch.empty(N, device="cuda"), max_norm=0.1)
        for ts in grads:
            for t in ts:
                room = torch.empty(0, dtype=t.dtype, device="cuda").set_(t.untyped_storage())
                assert (room[:gap] == 7).all() and (room[gap + t.numel():] == 7).all()


def test_many_tensors():
    """More than one launch's table, some ranks' tables cut in the middle."""
    N, T = 3, 700
    grads = gradients([5 + i % 37 for i in range(T)], ["bf16" if i % 3 else "f32" for i in range(T)], N)
    kept = [[t.clone() for t in ts] for ts in grads]
    for across in (True, False):
        norm = torch.empty(N, device="cuda")
        out = [[torch.empty_like(t) for t in ts] for ts in grads]
        vc.vc_clip_grad_norm(grads, norm, max_norm=1.0, out=out, across=across)
        check(grads, kept, norm, out, 1.0, across)


@pytest.mark.parametrize("n", [1, 7, 32768, 32769, 5000003])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_sizes(n, dt):
    grads = gradients([n], [dt], 2)
    kept = [[t.clone() for t in ts] for ts in grads]
    norm = [torch.empty((), device="cuda") for _ in range(2)]
    vc.vc_clip_grad_norm(grads, norm, max_norm=0.25)
    check(grads, kept, norm, grads, 0.25, True)


def test_nothing():
    norm = torch.full((2,), 7.0, device="cuda")
    vc.vc_clip_grad_norm([[], []], norm, max_norm=1.0)
    assert norm.tolist() == [0, 0]
    empty = [[torch.empty(0, device="cuda")], [torch.empty(0, device="cuda")]]
    norm.fill_(7)
    vc.vc_clip_grad_norm(empty, norm)
    assert norm.tolist() == [0, 0]


def test_infinity_nan_and_zeros():
    for bad, factor in ((math.inf, 0.0), (math.nan, math.nan)):
        grads = [[torch.ones(1000, device="cuda"), torch.ones(50, device="cuda").bfloat16()]]
        grads[0][0][77] = bad
        norm = torch.empty(1, device="cuda")
        vc.vc_clip_grad_norm(grads, norm, max_norm=1.0)
        assert (norm[0] == bad) if bad == math.inf else torch.isnan(norm[0])
        got = grads[0][1].float()
        assert (got == 0).all() if factor == 0 else torch.isnan(got).all()
        assert torch.isnan(grads[0][0][77])
    grads = [[torch.zeros(100, device="cuda")]]
    vc.vc_clip_grad_norm(grads, norm, max_norm=0.0)
    assert norm[0] == 0 and (grads[0][0] == 0).all()


def test_another_stream_a_graph_and_the_same_bits():
    grads, out = gradients([300000, 77], ["bf16", "f32"], 2), gradients([300000, 77], ["bf16", "f32"], 2, seed=1)
    norm = torch.empty(2, device="cuda")

    def go(stream=None):
        vc.vc_clip_grad_norm(grads, norm, max_norm=1.0, out=out, stream=stream)
    go()
    torch.cuda.synchronize()
    want = norm.clone(), [[t.clone() for t in ts] for ts in out]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for run in (lambda: go(side), graph.replay, graph.replay):
        norm.zero_()
        for ts in out:
            for t in ts:
                t.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert torch.equal(norm, want[0]) and all(torch.equal(a, b) for x, y in zip(out, want[1]) for a, b in zip(x, y))


def test_a_tensor_beyond_32_bits_of_elements():
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-5:], t[:3], t[2 ** 31 - 1:2 ** 31 + 2] = 3.0, 4.0, 2.0
    norm = torch.empty(1, device="cuda")
    vc.vc_clip_grad_norm([[t]], norm, max_norm=1.0)
    want = math.sqrt(5 * 9 + 3 * 16 + 3 * 4)
    assert abs(float(norm[0]) - want) <= NORM * want
    for at, v in ((n - 5, 3.0), (n - 1, 3.0), (0, 4.0), (2, 4.0), (2 ** 31 - 1, 2.0), (2 ** 31 + 1, 2.0), (2 ** 31 + 2, 0.0), (5, 0.0)):
        assert abs(float(t[at]) - v / want) <= store_bound(v / want, "bf16") * 1.001, at
