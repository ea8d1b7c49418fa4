"""Layer operators at the edges of their definitions: rows without elements,
and calls in a row that work in place on rows off 16-byte boundaries."""
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


@pytest.mark.parametrize("H", [1003, 1024])
def test_calls_in_place_one_after_another(H):
    """Each call reads what the one before wrote in place, rows of other blocks
    beside its own: enqueued at once, with the waits of one launch for the
    next on the GPU alone, the bits are those of calls that the host waits for."""
    N, rows, steps = 2, 1500, 12
    g = torch.Generator().manual_seed(H)
    send = (torch.randn(N, N * rows, H, generator=g) * 0.5).to(torch.bfloat16).cuda()
    start = torch.randn(N, rows, H, generator=g).to(torch.bfloat16).cuda()
    grad = torch.randn(N, rows, H, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    found = []
    for wait in (True, False, False):
        h, d, out = start.clone(), grad.clone(), torch.empty_like(start)
        rs = torch.empty(N, rows, device="cuda")
        dsend = torch.empty_like(send)
        torch.cuda.synchronize()
        for _ in range(steps):
            vc.vc_reduce_scatter_norm(send, w, out, residual=h, residual_out=h, rstd=rs)
            if wait:
                torch.cuda.synchronize()
            vc.vc_reduce_scatter_norm_backward(out, h, w, rs, dsend=dsend, dresidual=d, dresidual_out=d)
            if wait:
                torch.cuda.synchronize()
        found.append((h, d, out, dsend))
    for other in found[1:]:
        assert all(torch.equal(a, b) for a, b in zip(found[0], other))
