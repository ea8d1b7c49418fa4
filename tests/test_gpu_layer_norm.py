"""vc_reduce_scatter_norm and its backward on the GPU, against the definition
in 64 bits with bounds derived from the operations' roundings (layer_ref)."""
import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import layer_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(seed, N, rows, H, dt, shift=0):
    """Tensors whose buffers start `shift` elements off a 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)

    def make(*shape, by=1.0, plus=0.0):
        x = (torch.randn(*shape, generator=g) * by + plus).to(ref.DT[dt])
        raw = torch.zeros(x.numel() + 64, dtype=x.dtype, device="cuda")
        v = raw[shift:shift + x.numel()].view(*shape)
        v.copy_(x)
        return v

    return make(N, N * rows, H, by=N ** -0.5), make(N, rows, H, by=2.0), make(N, H, by=0.2, plus=1.0), make


def within(got, want, bound, what):
    off = np.abs(ref.f64(got) - want)
    assert np.all(off <= bound), (what, float((off - bound).max()), np.unravel_index((off - bound).argmax(), off.shape))


SIZES = [  # N, rows, H: one element, odd, a vector, more than one vector a thread, the longest rows, more rows than
    # blocks fit the GPU
    (1, 1, 1), (1, 3, 7), (2, 1, 8), (3, 2, 40), (8, 1, 4096), (2, 5, 1000), (4, 3, 2045), (1, 2, 8200),
    (2, 1, 16384), (1, 1, 32768), (2, 1, 40001), (1, 2, 12288), (1, 1, 12287), (3, 2, 16387),
    (3, 2, 10240), (3, 2, 5120), (1, 3000, 64), (2, 1500, 512), (2, 700, 5128), (1, 1, 49152), (64, 1, 64),
]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,rows,H", SIZES)
def test_forward(N, rows, H, dt):
    for shift in (0, 1):
        send, res, w, _ = inputs(N * rows + H, N, rows, H, dt, shift)
        out, rout = torch.empty_like(res), torch.empty_like(res)
        rstd = torch.empty(N, rows, device="cuda")
        vc.vc_reduce_scatter_norm(send, w, out, residual=res, residual_out=rout, rstd=rstd, eps=EPS)
        h, rs, y, dh, drs, dy = ref.norm(ref.f64(send), ref.f64(res), ref.f64(w), EPS)
        within(rout, h, dh + ref.store_bound(np.abs(h) + dh, dt), "residual_out")
        within(rstd, rs, drs, "rstd")
        within(out, y, dy + ref.store_bound(np.abs(y) + dy, dt), "out")
        # 8 bits: within half a step of y, and the step within its rounding of max|y| / 127
        q, scale = torch.empty(N, rows, H, dtype=torch.int8, device="cuda"), torch.empty(N, rows, device="cuda")
        vc.vc_reduce_scatter_norm(send, w, q, residual=res, scale=scale, eps=EPS)
        top = np.abs(y).max(-1)
        within(scale, top / 127, (dy.max(-1) + 4 * ref.U32 * top) / 127, "scale")
        step = ref.f64(scale)[..., None]
        off = np.abs(ref.f64(q) * step - y)
        assert np.all(off <= step * (0.5 + 1e-3) + 2 * dy), float((off / step).max())
        assert int(q.abs().amax(-1).min()) == 127 or float(top.min()) == 0


def test_lists_views_and_one_weight_for_all():
    """One tensor per rank, or a stacked tensor; a weight each, or one: the same bits."""
    N, rows, H = 3, 4, 136
    send, res, w, _ = inputs(1, N, rows, H, "bf16")
    w[1:] = w[0]
    a, b = torch.empty_like(res), [torch.empty(rows, H, dtype=torch.bfloat16, device="cuda") for _ in range(N)]
    vc.vc_reduce_scatter_norm(send, w, a, residual=res)
    vc.vc_reduce_scatter_norm(list(send), w[0].clone(), b, residual=[x.clone() for x in res])
    assert all(torch.equal(a[r], b[r]) for r in range(N))


@pytest.mark.parametrize("H", [512, 333])
def test_in_place_residual_and_no_residual(H):
    N, rows = 2, 3
    send, res, w, _ = inputs(2, N, rows, H, "bf16")
    want, sums = torch.empty_like(res), torch.empty_like(res)
    vc.vc_reduce_scatter_norm(send, w, want, residual=res, residual_out=sums)
    got, own = torch.empty_like(res), res.clone()
    vc.vc_reduce_scatter_norm(send, w, got, residual=own, residual_out=own)
    assert torch.equal(got, want) and torch.equal(own, sums)
    vc.vc_reduce_scatter_norm(send, w, got)
    vc.vc_reduce_scatter_norm(send, w, want, residual=torch.zeros_like(res))
    assert torch.equal(got, want)


@pytest.mark.parametrize("H", [256, 77])
def test_special_rows(H):
    """Zeros, NaN, infinity, and values whose 127 / max or square overflow."""
    N, rows = 1, 6
    x = torch.randn(N, rows, H)
    x[0, 0] = 0
    x[0, 1, 5] = float("nan")
    x[0, 2, 7] = float("inf")
    x[0, 3] *= 1e-38
    x[0, 4] *= 1e25
    x = x.cuda()
    w = torch.ones(H, device="cuda")
    out, rstd = torch.empty(N, rows, H, device="cuda"), torch.empty(N, rows, device="cuda")
    vc.vc_reduce_scatter_norm(x, w, out, rstd=rstd, eps=0.0)
    q, scale = torch.empty(N, rows, H, dtype=torch.int8, device="cuda"), torch.empty(N, rows, device="cuda")
    vc.vc_reduce_scatter_norm(x, w, q, scale=scale, eps=1.0)
    out, q, scale = out.cpu()[0], q.cpu()[0], scale.cpu()[0]
    assert torch.isnan(out[0]).all()  # 0 * 1/0
    assert scale[0] == 0 and not q[0].any()
    assert torch.isnan(out[1]).all() and torch.isnan(scale[1]) and not q[1].any()
    assert torch.isnan(out[2, 7]) and (out[2, :7] == 0).all() and torch.isnan(scale[2])
    # the smallest numbers: eps = 1 leaves the values as they are, 127 steps to the largest
    y = x.cpu()[0, 3].double()
    assert int(q[3].abs().max()) == 127
    assert (torch.round(y / (y.abs().max() / 127)) - q[3]).abs().max() <= 1
    assert (out[4] == 0).all() and scale[4] == 0  # its sum of squares is infinite in fp32
    assert torch.isfinite(out[5]).all() and scale[5] > 0


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,rows,H", [(1, 1, 1), (2, 3, 40), (3, 5, 333), (4, 67, 2048), (2, 700, 64), (1, 2, 16384),
                                      (1, 2, 12288), (2, 3, 8195), (1, 3, 20001), (2, 2, 49152)])
def test_backward(N, rows, H, dt):
    for shift in (0, 1):
        _, h, w, make = inputs(rows + H, N, rows, H, dt, shift)
        dout, dres = make(N, rows, H), make(N, rows, H)
        rstd = torch.rsqrt(h.float().square().mean(-1) + EPS)
        dsend, dresid = make(N, N * rows, H, by=0), make(N, rows, H, by=0)
        dw = torch.empty(N, H, device="cuda")
        vc.vc_reduce_scatter_norm_backward(dout, h, w, rstd, dsend=dsend, dresidual=dresid, dweight=dw,
                                           dresidual_out=dres)
        want, want_w, bound, bound_w = ref.norm_grad(ref.f64(dout), ref.f64(dres), ref.f64(h), ref.f64(w), ref.f64(rstd))
        within(dresid, want, bound + ref.store_bound(np.abs(want) + bound, dt), "dresidual")
        within(dw, want_w, bound_w, "dweight")
        for q in range(N):
            assert torch.equal(dsend[q], dresid.reshape(N * rows, H))
        # each alone, without dresidual_out, and in place
        alone, alone_w = torch.empty_like(dresid), torch.empty_like(dw)
        vc.vc_reduce_scatter_norm_backward(dout, h, w, rstd, dweight=alone_w)
        assert torch.equal(alone_w, dw)
        own = dres.clone()
        vc.vc_reduce_scatter_norm_backward(dout, h, w, rstd, dresidual=own, dresidual_out=own)
        assert torch.equal(own, dresid)
        vc.vc_reduce_scatter_norm_backward(dout, h, w, rstd, dresidual=alone)
        want, _, bound, _ = ref.norm_grad(ref.f64(dout), None, ref.f64(h), ref.f64(w), ref.f64(rstd))
        within(alone, want, bound + ref.store_bound(np.abs(want) + bound, dt), "dresidual alone")


@pytest.mark.parametrize("H", [96, 61])
def test_backward_against_differences(H):
    """<gradient, direction> against central differences of the 64-bit forward.

    With unit-size values and step e the truncation is e^2 / 6 times a third
    derivative of order one per element; e = 1e-4 leaves 1e-7 of the sum of
    magnitudes, far below the fp32 gradient's own bound times its size."""
    N, rows = 2, 3
    send, res, w, make = inputs(5, N, rows, H, "f32")
    rout, out, rstd = torch.empty_like(res), torch.empty_like(res), torch.empty(N, rows, device="cuda")
    vc.vc_reduce_scatter_norm(send, w, out, residual=res, residual_out=rout, rstd=rstd, eps=EPS)
    dout, dro = make(N, rows, H), make(N, rows, H)
    dsend, dres, dw = torch.empty_like(send), torch.empty_like(res), torch.empty(N, H, device="cuda")
    vc.vc_reduce_scatter_norm_backward(dout, rout, w, rstd, dsend=dsend, dresidual=dres, dweight=dw, dresidual_out=dro)
    base = [ref.f64(send), ref.f64(res), ref.f64(w)]

    def loss(a, b, c):
        h, _, y, *_ = ref.norm(a, b, c, EPS)
        return (y * ref.f64(dout)).sum() + (h * ref.f64(dro)).sum()

    rng = np.random.default_rng(0)
    for k, grad in enumerate((dsend, dres, dw)):
        for _ in range(3):
            v, e = rng.standard_normal(base[k].shape), 1e-4
            up, down = list(base), list(base)
            up[k], down[k] = base[k] + e * v, base[k] - e * v
            slope = (loss(*up) - loss(*down)) / (2 * e)
            terms = ref.f64(grad) * v
            assert abs(terms.sum() - slope) <= 2e-6 * np.abs(terms).sum(), (k, terms.sum(), slope)


def test_no_tokens():
    N, H = 2, 64
    e = torch.empty(N, 0, H, device="cuda")
    w = torch.ones(N, H, device="cuda")
    vc.vc_reduce_scatter_norm(e, w, torch.empty_like(e))
    dw = torch.full((N, H), 7.0, device="cuda")
    vc.vc_reduce_scatter_norm_backward(e, e, w, torch.empty(N, 0, device="cuda"), dweight=dw)
    assert not dw.any()


def test_another_stream_and_repeat_bits():
    N, rows, H = 4, 50, 2048
    send, res, w, make = inputs(9, N, rows, H, "bf16")
    h, rs = torch.empty_like(res), torch.empty(N, rows, device="cuda")
    out, dw = torch.empty_like(res), [torch.empty(N, H, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(2):
        vc.vc_reduce_scatter_norm(send, w, out, residual=res, residual_out=h, rstd=rs, stream=s)
        vc.vc_reduce_scatter_norm_backward(out, h, w, rs, dweight=dw[i], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(dw[0], dw[1])


def test_offsets_past_32_bits():
    """Send buffers of 2.4e9 elements: the last rows, from their own definition."""
    N, rows, H = 2, 25000, 49152
    send = torch.zeros(N, N * rows, H, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(N, H, device="cuda").to(torch.bfloat16)
    for q in range(N):
        send[q, -1] = last[q]
    out = torch.empty(N, rows, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    vc.vc_reduce_scatter_norm(send, w, out, eps=EPS)
    _, _, y, _, _, dy = ref.norm(ref.f64(last).reshape(2, 1, H).sum(0, keepdims=True), None, np.ones((1, H)), EPS)
    within(out[-1, -1].view(1, 1, H), y, 2 * dy + ref.store_bound(np.abs(y) + dy, "bf16"), "last row")
    assert not out[0, -1].any() and not out[-1, -2].any()
