"""Layer operators at the edges of their definitions: rows without elements."""
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dt", [torch.int8, torch.bfloat16, torch.float32])
def test_scales_move_without_rows(dt):
    """recv_scale takes scale for every slot, of rows of no elements too."""
    N, rows, k, cap = 2, 5, 2, 12
    g = torch.Generator().manual_seed(0)
    order = torch.randperm(N * cap, generator=g)[: N * rows * k].to(torch.int32)
    slots = order.view(N, rows, k).clone()
    slots[1, 2, 0] = -1
    scale, got = torch.rand(N, rows, generator=g).cuda(), torch.full((N, cap), -1.0, device="cuda")
    want = got.cpu().view(-1)
    for a, s in enumerate(slots.view(-1).tolist()):
        if s >= 0:
            want[s] = scale.cpu().view(-1)[a // k]
    send, recv = torch.empty(N, rows, 0, dtype=dt, device="cuda"), torch.empty(N, cap, 0, dtype=dt, device="cuda")
    vc.vc_dispatch(send, slots.cuda(), recv)
    vc.vc_dispatch(send, slots.cuda(), recv, scale=scale, recv_scale=got)
    assert torch.equal(got.cpu().view(-1), want)
