"""Layer operators at the edges of their definitions: rows without elements,
8-bit rounding at half steps and of the smallest numbers, and calls in a row that work in place on rows off 16-byte boundaries."""
import numpy as np
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


@pytest.mark.parametrize("H", [256, 1001])
def test_eight_bits_are_the_documented_product(H):
    """out = y times fp32's 127 / max |y|, rounded once to the nearest even
    whole number, with y as the same call in fp32 gives it: the product of two
    fp32 numbers is exact in 64 bits.  Rows on a grid of half steps (127 / max
    = 1), ordinary ones, subnormal ones, one with an infinity and one with a
    NaN (eps = 1 and a weight of 1 leave small rows as they are; on the grid
    the weight makes up for rms)."""
    rows = 64
    g = torch.Generator().manual_seed(H)
    x = torch.randn(1, rows, H, generator=g)
    x[0, 8:16] *= 1e-30
    x[0, 16:24] *= 1e-38
    x[0, 24:32] *= 1e-41
    x[0, 32:40] = torch.randint(-254, 255, (8, H), generator=g).float() / 2
    x[0, 32:40, 3] = 127
    x[0, 40, 5], x[0, 41, 5] = float("inf"), float("nan")
    x = x.cuda()
    w = torch.ones(1, H, device="cuda")
    y = torch.empty(1, rows, H, device="cuda")
    q, scale = torch.empty(1, rows, H, dtype=torch.int8, device="cuda"), torch.empty(1, rows, device="cuda")
    vc.vc_reduce_scatter_norm(x, w, y, eps=1.0)
    vc.vc_reduce_scatter_norm(x, w, q, scale=scale, eps=1.0)
    y, q, scale = y.cpu().numpy()[0], q.cpu().numpy()[0], scale.cpu().numpy()[0]
    top = np.abs(y).max(-1)
    assert np.array_equal(scale, top / np.float32(127), equal_nan=True)
    for t in range(rows):
        if not np.isfinite(top[t]):
            assert t in (40, 41) and not q[t].any()
        elif top[t] > 1e-30:
            inv = np.float32(127) / top[t]
            assert np.array_equal(q[t], np.rint(y[t].astype(np.float64) * np.float64(inv))), t
        else:  # 127 / max would overflow for the smallest: both are taken 2^64 times as large
            inv = np.float32(127) / (top[t] * np.float32(2.0 ** 64))
            assert np.array_equal(q[t], np.rint(y[t].astype(np.float64) * 2.0 ** 64 * np.float64(inv))), t
            assert np.abs(q[t].astype(int)).max() == 127
    assert (scale[24:32] < 2.0 ** -126).all()
    # a row whose y are whole and half numbers up to 127: the ties go to even numbers
    w = (x[:, 32].square().mean(-1) + 1.0).sqrt()
    one = x[:, 32:33].clone()
    vc.vc_reduce_scatter_norm(one, w.expand(H).contiguous(), y32 := torch.empty_like(one), eps=1.0)
    vc.vc_reduce_scatter_norm(one, w.expand(H).contiguous(), q8 := torch.empty(1, 1, H, dtype=torch.int8, device="cuda"),
                              scale=torch.empty(1, 1, device="cuda"), eps=1.0)
    v = y32.cpu().numpy()[0, 0]
    inv = np.float32(127) / np.abs(v).max()
    assert np.array_equal(q8.cpu().numpy()[0, 0], np.rint(v.astype(np.float64) * np.float64(inv)))


def test_infinite_values_without_a_nan():
    """An infinite weight, on values that are not 0: scale infinity and zeros."""
    H = 64
    x, w = torch.randn(1, 2, H).abs().add(0.5).cuda(), torch.ones(1, H, device="cuda")
    w[0, 7] = float("inf")
    q, scale = torch.empty(1, 2, H, dtype=torch.int8, device="cuda"), torch.empty(1, 2, device="cuda")
    vc.vc_reduce_scatter_norm(x, w, q, scale=scale)
    assert torch.isinf(scale).all() and not q.any()
