"""vc_dispatch_plan, vc_dispatch, vc_combine and its backward on the GPU.

Plans and moved rows are compared exactly; sums with the 64-bit definition,
within the roundings of topk fp32 products and additions and the last store.
"""
import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make_plan(ids, E, cap):
    N = ids.shape[0]
    slots = torch.full_like(ids, -7)
    offsets = torch.full((N, E // N + 1), -7, dtype=torch.int32, device="cuda")
    vc.vc_dispatch_plan(ids, slots, offsets, cap)
    return slots, offsets


def some_ids(seed, N, rows, k, E, lo=-1):
    """Ids of [lo, E], so -1 and E, which are nobody's, among them."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, E + 1, (N, rows, k), generator=g, dtype=torch.int32).cuda()


PLANS = [  # N, rows, k, E, capacity: one choice, one warp's worth, more than one step of a warp, all cluster sizes, shared memory about 48 KB
    (1, 1, 1, 1, 1), (1, 5, 2, 3, 100), (2, 1, 4, 8, 3), (8, 4, 4, 64, 16), (3, 33, 5, 33, 40), (4, 100, 6, 128, 170),
    (8, 63, 8, 256, 500), (2, 1025, 2, 1024, 2000), (8, 500, 8, 64, 700), (5, 3000, 3, 20, 1800), (64, 70, 8, 1024, 70),
    (1, 20000, 6, 7, 30000), (1, 90, 4, 341, 200), (1, 90, 4, 342, 200),
]


@pytest.mark.parametrize("N,rows,k,E,cap", PLANS)
def test_plan(N, rows, k, E, cap):
    ids = some_ids(rows, N, rows, k, E)
    slots, offsets = make_plan(ids, E, cap)
    want_s, want_o = ref.plan(ids.cpu().numpy(), E, cap)
    assert np.array_equal(slots.cpu().numpy(), want_s)
    assert np.array_equal(offsets.cpu().numpy(), want_o)


@pytest.mark.parametrize("which", ["none", "one", "outside"])
def test_plan_of_one_sided_choices(which):
    """Nobody chooses, everybody chooses one expert, ids far outside."""
    N, rows, k, E, cap = 4, 700, 4, 16, 64
    ids = torch.full((N, rows, k), {"none": -1, "one": 9, "outside": 2 ** 31 - 1}[which], dtype=torch.int32, device="cuda")
    if which == "outside":
        ids[:, ::2] = -2 ** 31
    slots, offsets = make_plan(ids, E, cap)
    want_s, want_o = ref.plan(ids.cpu().numpy(), E, cap)
    assert np.array_equal(slots.cpu().numpy(), want_s) and np.array_equal(offsets.cpu().numpy(), want_o)


def test_plan_of_no_tokens():
    ids = torch.empty(2, 0, 3, dtype=torch.int32, device="cuda")
    slots, offsets = make_plan(ids, 8, 4)
    assert not offsets.any()


ROWS = [  # N, rows, k, E, cap, H: short and long rows, odd rows, more than one piece a row
    (1, 1, 1, 1, 1, 1), (2, 3, 2, 4, 5, 16), (3, 17, 3, 6, 20, 33), (8, 4, 4, 64, 16, 512), (5, 77, 3, 20, 60, 1003),
    (4, 50, 8, 32, 130, 2056), (1, 9, 32, 64, 300, 4099), (64, 2, 2, 64, 8, 24),
]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}


def values(g, dt, *shape):
    if dt == "i8":
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()
    return torch.randn(*shape, generator=g).to(TYPES[dt]).cuda()


def shifted(x, shift):
    """x's values in a buffer that starts `shift` elements off a 16-byte boundary."""
    raw = torch.zeros(x.numel() + shift, dtype=x.dtype, device="cuda")
    v = raw[shift:].view(x.shape)
    v.copy_(x)
    return v


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16", "i8"])
@pytest.mark.parametrize("N,rows,k,E,cap,H", ROWS)
def test_dispatch(N, rows, k, E, cap, H, dt):
    g = torch.Generator().manual_seed(H)
    ids = some_ids(H, N, rows, k, E)
    slots, _ = make_plan(ids, E, cap)
    sl = slots.cpu().numpy().reshape(-1)
    for shift in (0, 1):
        send, recv = shifted(values(g, dt, N, rows, H), shift), shifted(values(g, dt, N, cap, H), 5 * shift)
        scale, rscale = torch.rand(N, rows, device="cuda"), torch.full((N, cap), -1.0, device="cuda")
        want, want_s = recv.cpu().clone().view(-1, H), rscale.cpu().clone().view(-1)
        for a in np.nonzero(sl >= 0)[0]:
            want[sl[a]] = send.view(-1, H)[a // k].cpu()
            want_s[sl[a]] = scale.view(-1)[a // k].cpu()
        vc.vc_dispatch(send, slots, recv, scale=scale, recv_scale=rscale)
        assert torch.equal(recv.cpu().view(-1, H), want) and torch.equal(rscale.cpu().view(-1), want_s)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,rows,k,E,cap,H", ROWS)
def test_combine_and_backward(N, rows, k, E, cap, H, dt):
    g = torch.Generator().manual_seed(H + 1)
    ids = some_ids(H, N, rows, k, E)
    slots, _ = make_plan(ids, E, cap)
    sl = slots.cpu().numpy().reshape(-1, k)
    on = sl >= 0
    for shift in (0, 1):
        recv, out = shifted(values(g, dt, N, cap, H), shift), shifted(values(g, dt, N, rows, H), 3 * shift)
        w = torch.rand(N, rows, k, generator=g).cuda()
        # rows and weights that no slot takes are never looked at
        w.view(-1, k)[torch.from_numpy(~on).cuda()] = float("nan")
        free = np.ones(N * cap, bool)
        free[sl[on]] = False
        recv.view(-1, H)[torch.from_numpy(free).cuda()] = float("nan")
        y = ref.f64(recv).reshape(-1, H)[np.maximum(sl, 0)]
        for weights in (w, None):
            vc.vc_combine(recv, slots, out, weights=weights)
            w64 = np.where(on, 1.0 if weights is None else ref.f64(w).reshape(-1, k), 0.0)
            terms = np.where(on[..., None], w64[..., None] * np.where(on[..., None], y, 0.0), 0.0)
            want, size = terms.sum(1), np.abs(terms).sum(1)
            bound = (k + 2) * ref.U32 * size + ref.store_bound(size * (1 + 1e-5), dt)
            off = np.abs(ref.f64(out).reshape(-1, H) - want)
            assert np.all(off <= bound), (weights is None, float((off - bound).max()))
        # backward
        dout = shifted(values(g, dt, N, rows, H), shift)
        drecv = shifted(values(g, dt, N, cap, H), 2 * shift)
        before = drecv.clone()
        dw = torch.full((N, rows, k), -7.0, device="cuda")
        vc.vc_combine_backward(dout, recv, slots, weights=w, drecv=drecv, dweights=dw)
        d64 = ref.f64(dout).reshape(-1, H)
        got = ref.f64(drecv).reshape(-1, H)
        prods = np.where(on[..., None], d64[:, None, :] * np.where(on[..., None], y, 0.0), 0.0)
        off = np.abs(ref.f64(dw).reshape(-1, k) - prods.sum(-1))
        assert np.all(off <= (H + 8) * ref.U32 * np.abs(prods).sum(-1)), float(off.max())
        t, j = np.nonzero(on)
        want = w64_of(w, k)[t, j][:, None] * d64[t]
        off = np.abs(got[sl[t, j]] - want)
        assert np.all(off <= 2 * ref.U32 * np.abs(want) + ref.store_bound(want, dt))
        keep = torch.from_numpy(free).cuda()
        assert torch.equal(drecv.view(-1, H)[keep], before.view(-1, H)[keep])
        # each alone
        one, two = before.clone(), torch.empty_like(dw)
        vc.vc_combine_backward(dout, None, slots, weights=w, drecv=one)
        vc.vc_combine_backward(dout, recv, slots, weights=w, dweights=two)
        assert torch.equal(one, drecv) and torch.equal(two, dw)


def w64_of(w, k):
    return ref.f64(w).reshape(-1, k)


def test_combine_backward_against_differences():
    """Combine is linear in its rows and in its weights, so a difference of
    the 64-bit form along any direction is exact but for 64-bit rounding; the
    fp32 gradients are within 1e-5 of the magnitudes (64 terms)."""
    N, rows, k, E, cap, H = 2, 6, 3, 4, 12, 64
    g = torch.Generator().manual_seed(3)
    slots, _ = make_plan(some_ids(4, N, rows, k, E), E, cap)
    recv, dout, w = values(g, "f32", N, cap, H), values(g, "f32", N, rows, H), torch.rand(N, rows, k, generator=g).cuda()
    drecv, dw = torch.zeros_like(recv), torch.empty_like(w)
    vc.vc_combine_backward(dout, recv, slots, weights=w, drecv=drecv, dweights=dw)
    sl = slots.cpu().numpy().reshape(-1, k)

    def loss(y, ww):
        rows_ = np.where((sl >= 0)[..., None], y.reshape(-1, H)[np.maximum(sl, 0)], 0.0)
        return ((rows_ * ww.reshape(-1, k, 1)).sum(1) * ref.f64(dout).reshape(-1, H)).sum()

    rng = np.random.default_rng(1)
    base = [ref.f64(recv), ref.f64(w)]
    for i, grad in enumerate((drecv, dw)):
        v = rng.standard_normal(base[i].shape)
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + 0.5 * v, base[i] - 0.5 * v
        terms = ref.f64(grad) * v
        assert abs(loss(*up) - loss(*down) - terms.sum()) <= 1e-5 * np.abs(terms).sum()


def test_slots_outside_are_skipped():
    N, rows, k, cap, H = 2, 4, 2, 8, 40
    slots = torch.full((N, rows, k), N * cap, dtype=torch.int32, device="cuda")
    slots[1] = -2 ** 31
    slots[0, 0, 0] = N * cap - 1
    send, recv = torch.randn(N, rows, H, device="cuda"), torch.zeros(N, cap, H, device="cuda")
    vc.vc_dispatch(send, slots, recv)
    assert torch.equal(recv[1, -1], send[0, 0]) and int(recv.ne(0).any(-1).sum()) == 1
    out = torch.empty_like(send)
    vc.vc_combine(recv, slots, out)
    assert torch.equal(out[0, 0], send[0, 0]) and int(out.ne(0).any(-1).sum()) == 1


def test_dispatch_is_undone_by_combine_without_weights():
    """combine(dispatch(x)) without weights = x times the choices taken: dispatch's gradient."""
    N, rows, k, E, cap, H = 4, 30, 4, 16, 400, 256
    slots, _ = make_plan(some_ids(2, N, rows, k, E), E, cap)
    x = torch.randint(-99, 99, (N, rows, H), device="cuda").float()  # whole numbers: sums are exact
    recv = torch.zeros(N, cap, H, device="cuda")
    vc.vc_dispatch(x, slots, recv)
    out = torch.empty_like(x)
    vc.vc_combine(recv, slots, out)
    assert torch.equal(out, x * (slots >= 0).sum(-1, keepdim=True))


def test_offsets_past_32_bits():
    """Receive buffers of 2.3e9 elements: rows at their far ends."""
    N, rows, k, cap, H = 2, 3, 2, 70000, 32768
    recv = torch.zeros(N, cap, H, dtype=torch.float16, device="cuda")
    slots = torch.tensor([[[cap - 1, 2 * cap - 1], [0, cap], [cap - 2, -1]], [[cap + 5, -1], [-1, -1], [7, 9]]],
                         dtype=torch.int32, device="cuda")
    x = torch.randn(N, rows, H, device="cuda").half()
    vc.vc_dispatch(x, slots, recv)
    assert torch.equal(recv[0, -1], x[0, 0]) and torch.equal(recv[1, -1], x[0, 0]) and torch.equal(recv[0, -2], x[0, 2])
    out = torch.empty_like(x)
    vc.vc_combine(recv, slots, out)
    assert torch.equal(out[0, 0], x[0, 0] + x[0, 0]) and torch.equal(out[0, 2], x[0, 2]) and not out[1, 1].any()
    drecv, dw = torch.zeros_like(recv), torch.empty(N, rows, k, device="cuda")
    vc.vc_combine_backward(x, recv, slots, drecv=drecv, dweights=dw)
    assert torch.equal(drecv[1, -1], x[0, 0]) and torch.equal(drecv[0, -1], x[0, 0])
    want = (x[0, 0].double() ** 2).sum()
    assert abs(float(dw[0, 0, 1]) - float(want)) <= 1e-4 * float(want)


def test_a_layer_in_a_graph_on_another_stream():
    """Route, plan, dispatch and combine captured and replayed with new inputs."""
    N, rows, k, E, cap, H = 4, 16, 2, 8, 128, 128
    logits, x = torch.randn(N, rows, E, device="cuda"), torch.randn(N, rows, H, device="cuda")
    ids = torch.empty(N, rows, k, dtype=torch.int32, device="cuda")
    w = torch.empty(N, rows, k, device="cuda")
    slots, offsets = torch.empty_like(ids), torch.empty(N, E // N + 1, dtype=torch.int32, device="cuda")
    recv, out = torch.zeros(N, cap, H, device="cuda"), torch.empty_like(x)

    def layer():
        vc.vc_route(logits, ids, w)
        vc.vc_dispatch_plan(ids, slots, offsets, cap)
        vc.vc_dispatch(x, slots, recv)
        vc.vc_combine(recv, slots, out, weights=w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for _ in range(2):
        x.copy_(torch.randn_like(x))
        logits.copy_(torch.randn_like(logits))
        g.replay()
        # every choice was taken, and the weights sum to 1: the tokens come back
        torch.cuda.synchronize()
        assert bool((slots >= 0).all())
        assert (out - x).abs().max() <= 1e-6 * x.abs().max()
