"""The lists that vc_clip_grad_norm takes: the compiled pass over them gives what
asking each tensor in Python gives, leaves alone what it cannot read, and costs
less than the work."""
import time

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc
from collective_communication_algorithms_virtual_gb300 import binding

from .test_gpu_clip import MIXED, check, gpu, gradients  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_same_arrays():
    for N in (1, 3):
        grads, out = gradients(*MIXED, N, gap=1), gradients(*MIXED, N, seed=1)
        for a, b in ((grads, None), (grads, out), (grads, grads), (tuple(map(tuple, grads)), out), ([[]] * N, None)):
            want = binding._gradients(a, b, N, len(a[0]), 0)
            assert binding._lists().pack(a, b, 0) == want
    t = torch.nn.Parameter(torch.ones(5, device="cuda"))
    assert binding._lists().pack([[t]], None, 0) == binding._gradients([[t]], None, 1, 1, 0)


class Sub(torch.Tensor):
    pass


def test_other_lists_are_left_to_python():
    f, h = torch.ones(8, device="cuda"), torch.ones(8, device="cuda", dtype=torch.bfloat16)
    pack = binding._lists().pack
    assert pack([[f, h], [f, h]], [[f, h], [f, h]], 0) is not None
    for grads, out in (([], None), ([[f, h], [f]], None), ([[f], [h]], None), ([[f.cpu()]], None), ([[f[::2]]], None),
                       ([[None]], None), ([[f.double()]], None), ([[f.as_subclass(Sub)]], None), ([iter([f])], None),
                       (f, None), ([[f]], [[h]]), ([[f]], [[f[:4]]]), ([[f]], [[f], [f]]), ([[f]], [[]]), ([[f]], f),
                       ([[f.to_sparse()]], None), ([[torch.empty(3, device="meta")]], None)):
        assert pack(grads, out, 0) is None
    assert pack([[f]], None, 1) is None


def test_subclasses_still_work():
    grads = gradients(*MIXED, 2)
    kept = [[t.clone() for t in ts] for ts in grads]
    norm = torch.empty(2, device="cuda")
    vc.vc_clip_grad_norm([[t.as_subclass(Sub) for t in ts] for ts in grads], norm, max_norm=0.5)
    check(grads, kept, norm, grads, 0.5, True)


@pytest.mark.parametrize("bad", ["type", "device", "size", "stride", "ranks"])
def test_refusals_on_the_gpu(bad):
    f = lambda: torch.ones(8, device="cuda")  # noqa: E731
    out = {"type": [[f()], [f().bfloat16()]], "device": [[f()], [f().cpu()]], "size": [[f()], [f()[:4]]],
           "stride": [[f()], [torch.ones(16, device="cuda")[::2]]], "ranks": [[f()]]}[bad]
    with pytest.raises(vc.VCError):
        vc.vc_clip_grad_norm([[f()], [f()]], torch.empty(2, device="cuda"), max_norm=1.0, out=out)


def test_small_tensors_cost_less_than_asking_each():
    """2048 tensors and as many outputs; asked one by one in Python they took 0.6
    us each."""
    N, T = 8, 256
    grads, out = ([[torch.ones(64, device="cuda") for _ in range(T)] for _ in range(N)] for _ in range(2))
    norm, best = torch.empty(N, device="cuda"), 1.0
    for _ in range(30):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        vc.vc_clip_grad_norm(grads, norm, max_norm=1.0, out=out)
        best = min(best, time.perf_counter() - begin)
    assert best / (N * T) < 0.3e-6
