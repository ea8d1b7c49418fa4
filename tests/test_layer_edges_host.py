"""Arguments at the edges that the layer operators' binding refuses, on the CPU."""
import pytest
import torch

from collective_communication_algorithms_virtual_gb300 import binding as b

from .test_binding_checks import Recorder
from .test_layer_host import Fake

I = torch.int32


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(b, "lib", lambda: r)
    monkeypatch.setattr(b, "CHECK_TENSORS", True)
    return r


def refused(rec, call):
    with pytest.raises(b.VCError) as e:
        call()
    assert e.value.status == b.VC_ERR_INVALID_ARG
    assert rec.calls == []


@pytest.mark.parametrize("none", [[], ()])
@pytest.mark.parametrize("call", [
    lambda no: b.vc_reduce_scatter_norm(no, Fake(8), Fake(2, 3, 8), stream=1),
    lambda no: b.vc_reduce_scatter_norm(Fake(2, 6, 8), Fake(8), no, stream=1),
    lambda no: b.vc_reduce_scatter_norm(Fake(2, 6, 8), no, Fake(2, 3, 8), stream=1),
    lambda no: b.vc_reduce_scatter_norm_backward(no, no, Fake(8), no, dweight=no, stream=1),
    lambda no: b.vc_route(no, no, no, stream=1),
    lambda no: b.vc_route(Fake(2, 3, 16), no, Fake(2, 3, 4), stream=1),
    lambda no: b.vc_route_backward(no, no, no, no, stream=1),
    lambda no: b.vc_dispatch_plan(no, no, no, 12, stream=1),
    lambda no: b.vc_dispatch_plan(Fake(2, 3, 4, dtype=I), Fake(2, 3, 4, dtype=I), no, 12, stream=1),
    lambda no: b.vc_dispatch(no, no, no, stream=1),
    lambda no: b.vc_dispatch(Fake(2, 3, 8), Fake(2, 3, 4, dtype=I), no, stream=1),
    lambda no: b.vc_combine(no, no, no, stream=1),
    lambda no: b.vc_combine_backward(no, no, no, stream=1),
])
def test_no_tensors_are_refused(rec, call, none):
    refused(rec, lambda: call(none))


@pytest.mark.parametrize("over", [dict(scale=1e39), dict(scale=-1e300), dict(ngroups=1 << 31), dict(group_top=-1 << 40),
                                  dict(topk_groups=1.5), dict(score=1 << 32)])
def test_route_numbers_that_the_library_cannot_hold_are_refused(rec, over):
    """A scale that is finite here and infinite in fp32, numbers past int32, a
    count that is not whole."""
    refused(rec, lambda: b.vc_route(Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 4), stream=1, **over))
    over = {k: v for k, v in over.items() if k in ("scale", "score")}
    if over:
        refused(rec, lambda: b.vc_route_backward(Fake(2, 3, 4), Fake(2, 3, 16), Fake(2, 3, 4, dtype=I), Fake(2, 3, 16),
                                                 stream=1, **over))
