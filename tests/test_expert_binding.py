"""Arguments of the experts' operators that are no tensors, on the CPU: refused
with VCError like any other wrong argument."""
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .test_expert_host import on0, recorded  # noqa: F401

INVALID = 1


def refused(call, **args):
    with pytest.raises(vc.VCError) as e:
        call(**args)
    assert e.value.status == INVALID


def test_an_empty_list_of_gradients(recorded):  # noqa: F811
    x, w, off, out = on0(2, 4, 8), on0(2, 3, 8, 6), on0(2, 4, dtype=torch.int32), on0(2, 4, 6)
    good = dict(dout=out, rows=x, weight=w, offsets=off, drows=on0(2, 4, 8), dweight=on0(2, 3, 8, 6))
    vc.vc_expert_product_backward(**good)
    for name in ("dweight", "drows", "rows", "dout", "offsets"):
        refused(vc.vc_expert_product_backward, **{**good, name: []})
    refused(vc.vc_expert_product_backward, **{**good, "drows": None, "dweight": []})


@pytest.mark.parametrize("grads", [[[None]], [[on0(4), None]], [[on0(4), 3.0]], on0(1, 2, 4), None, [on0(1)[0]], [None], [[on0(4)], None],
                                   iter([[on0(4)]])])
def test_gradients_that_are_no_lists_of_tensors(recorded, grads):  # noqa: F811
    refused(vc.vc_clip_grad_norm, grads=grads, norm=on0(1 if not isinstance(grads, list) else len(grads)))
    assert not recorded


@pytest.mark.parametrize("out", [[[None]], [None], [on0(1)[0]], 3, [[on0(4)], None], []])
def test_outputs_that_are_no_lists_of_tensors(recorded, out):  # noqa: F811
    refused(vc.vc_clip_grad_norm, grads=[[on0(4)]], norm=on0(1), max_norm=1.0, out=out)
    assert not recorded


def test_a_rank_of_one_tensor_is_its_rows(recorded):  # noqa: F811
    vc.vc_clip_grad_norm([on0(2, 4)], on0(1), max_norm=1.0, out=[on0(2, 4)])
    assert recorded[-1][1][4:6] == (1, 2)


@pytest.mark.parametrize("check", [True, False])
def test_ranks_of_tuples_are_lists(recorded, monkeypatch, check):  # noqa: F811
    monkeypatch.setattr(vc.binding, "CHECK_TENSORS", check)
    vc.vc_clip_grad_norm(((on0(4), on0(2)),), on0(1), max_norm=1.0, out=((on0(4), on0(2)),))
    assert recorded[-1][1][4:6] == (1, 2)


def test_the_drill_wants_somewhere_to_write():
    assert vc.lib().vc_product_selftest(None, None) == INVALID
