"""The rounding to 8 bits by blocks, bit for bit as it is documented, and the
products of such rows and weights against 64-bit products of the values they
stand for, within bounds derived in tests/expert_ref.py."""
import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import expert_ref as ref
from .layer_ref import DT, f64, store_bound

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def blocks(n):
    return -(-n // 128)


def quantized(x, B):
    """x (rows, width) fp32 -> e4m3 codes and scales, in fp32 operations as vc.h has them."""
    rows, width = x.shape
    codes, scales = np.zeros(x.shape, np.uint8), np.zeros((-(-rows // B), blocks(width)), np.float32)
    with np.errstate(all="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                part = x[i * B:(i + 1) * B, j * 128:(j + 1) * 128]
                most = np.abs(part).max()  # NaN where there is one
                if not np.isfinite(most):
                    scales[i, j] = most
                    continue
                scales[i, j] = max(most / np.float32(448), np.float32(2.0 ** -126)) if most else 0
                q = part * min(np.float32(448) / most, np.float32(2.0 ** 126))
                codes[i * B:(i + 1) * B, j * 128:(j + 1) * 128] = \
                    torch.from_numpy(np.clip(q, -448, 448)).to(F8).view(torch.uint8).numpy()
    return codes, scales


def check_quantized(x, out, scale, B, last=None):
    for r in range(len(x)):
        mats = [(x[r], out[r], scale[r])] if x[r].dim() == 2 else zip(x[r], out[r], scale[r])
        for a, q, s in mats:
            n = a.shape[0] if last is None else last[r]
            codes, scales = quantized(a[:n].float().cpu().numpy(), B)
            got = q.view(torch.uint8).cpu().numpy()
            # a zero's sign aside
            assert np.array_equal(np.where(got[:n] == 0x80, 0, got[:n]), np.where(codes == 0x80, 0, codes))
            m = scales.shape[0]
            assert np.array_equal(s[:m].cpu().numpy(), scales, equal_nan=True)
            if last is not None:  # behind the last row: as they were
                assert (got[n:] == 0x5a).all() and (s[n:] == 7).all()


def filled(shape, dt, g, shift=0):
    n = int(np.prod(shape[1:], dtype=np.int64))
    out = []
    for _ in range(shape[0]):
        t = torch.zeros(n + shift + 8, dtype=DT[dt], device="cuda")[shift:shift + n].view(shape[1:])
        t.copy_(torch.randn(*shape[1:], generator=g, device="cuda") * torch.exp(2 * torch.randn(*shape[1:-1], 1, generator=g, device="cuda")))
        out.append(t)
    return out


def room(shape, dtype, fill, shift=0):
    n = int(np.prod(shape[1:], dtype=np.int64))
    out = []
    for _ in range(shape[0]):
        t = torch.full((n + shift + 8,), fill, dtype=torch.uint8 if dtype is F8 else dtype, device="cuda")
        out.append(t[shift:shift + n].view(shape[1:]).view(dtype) if dtype is F8 else t[shift:shift + n].view(shape[1:]))
    return out


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape,shift", [((2, 5, 256), 0), ((1, 1, 128), 0), ((3, 33, 1000), 0), ((2, 7, 129), 0), ((1, 9, 1), 0),
                                         ((2, 4, 4104), 0), ((2, 6, 640), 1), ((1, 300, 72), 3), ((64, 2, 136), 0)])
@pytest.mark.parametrize("B", [1, 128])
def test_quantize(dt, shape, shift, B):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = filled(shape, dt, g, shift)
    out, scale = room(shape, F8, 0x5a, shift), room((shape[0], -(-shape[1] // B), blocks(shape[2])), torch.float32, 7)
    vc.vc_quantize_fp8(x, out, scale, block_rows=B)
    check_quantized(x, out, scale, B)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_matrices(dt):
    g = torch.Generator(device="cuda").manual_seed(2)
    for rows, width in ((256, 384), (130, 200), (1, 128), (129, 7)):
        x = filled((2, 3, rows, width), dt, g)
        for B in (1, 128):
            out, scale = room((2, 3, rows, width), F8, 0x5a), room((2, 3, -(-rows // B), blocks(width)), torch.float32, 7)
            vc.vc_quantize_fp8(x, out, scale, block_rows=B)
            check_quantized(x, out, scale, B)


def test_quantize_received_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = filled((3, 40, 264), "bf16", g)
    off = torch.tensor([[0, 3, 17], [0, 0, 0], [0, 30, 40]], dtype=torch.int32, device="cuda")
    out, scale = room((3, 40, 264), F8, 0x5a), room((3, 40, 3), torch.float32, 7)
    vc.vc_quantize_fp8(x, out, scale, offsets=off)
    check_quantized(x, out, scale, 1, last=[17, 0, 40])


def test_quantize_the_ends_of_the_range():
    """Zeros, the smallest and largest numbers, NaN and infinities, each in a block of its own."""
    x = torch.randn(12, 256, device="cuda")
    x[0] = 0
    x[1, :128], x[2, 128:] = 1e-45, 1e-40
    x[3, 5], x[4, 200], x[5, 3], x[5, 4] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[6], x[7, 0], x[8] = 3e38, -torch.finfo(torch.float32).max, 5e-39
    x[9, :128], x[10] = 2.0 ** -118, -0.0
    for B in (1, 128):
        out, scale = room((1, 12, 256), F8, 0x5a), room((1, 12 if B == 1 else 1, 2), torch.float32, 7)
        vc.vc_quantize_fp8([x], out, scale, block_rows=B)
        check_quantized([x], out, scale, B)


def values(q, scale, B):
    s = np.repeat(f64(scale), 128, -1)[..., :q.shape[-1]]
    if B == 128:
        s = np.repeat(s, 128, -2)[..., :q.shape[-2], :]
    return q.to(torch.float32).double().cpu().numpy() * s


def product(dt, rows, cap, win, width, shift=0):
    N, each = np.asarray(rows).shape
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = filled((N, cap, win), "bf16", g), filled((N, each, width, win), "bf16", g)
    ends = np.concatenate([np.zeros((N, 1), np.int64), np.cumsum(rows, 1)], 1).astype(np.int32)
    off = torch.from_numpy(ends).cuda()
    x8, xs = room((N, cap, win), F8, 0x7f, shift), room((N, cap, blocks(win)), torch.float32, float("nan"))
    w8, ws = room((N, each, width, win), F8, 0, shift), room((N, each, blocks(width), blocks(win)), torch.float32, 0)
    vc.vc_quantize_fp8(x, x8, xs, offsets=off)
    vc.vc_quantize_fp8(w, w8, ws, block_rows=128)
    out = room((N, cap, width), DT[dt], 7, shift)
    vc.vc_expert_product_fp8(x8, xs, w8, ws, off, out)
    assert vc.vc_device_errors() == 0
    for d in range(N):
        n = ends[d, -1]
        assert (out[d][n:] == 7).all()
        X, W = values(x8[d][:n], xs[d][:n], 1), values(w8[d], ws[d], 128)
        for i in range(each):
            lo, hi = ends[d, i], ends[d, i + 1]
            want, size = X[lo:hi] @ W[i].T, np.abs(X[lo:hi]) @ np.abs(W[i]).T
            # a block's scale is rounded once, its sums are added by one rounding each
            bound = (win + 2 * blocks(win) + 2) * ref.ULP * size + store_bound(want, dt)
            got = f64(out[d][lo:hi])
            ok = np.abs(got - want) <= bound
            if dt == "f16":  # 65520 and above round to infinity
                ok |= (np.abs(want) + bound >= 65520) & (got == np.copysign(np.inf, want))
            assert ok.all(), (d, i)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("win,width", [(128, 256), (512, 128), (64, 16), (4096, 272), (1000, 515), (1, 1), (129, 384), (272, 640)])
def test_product(dt, win, width):
    product(dt, [[17, 130, 0], [1, 257, 33], [0, 0, 300]], 301, win, width)


@pytest.mark.parametrize("rows,cap", [([[1]], 1), ([[0, 0]], 5), ([[128, 128]], 256), ([[700, 3]], 900), ([[1] * 16] * 64, 20)])
def test_product_rows(rows, cap):
    product("bf16", rows, cap, 264, 264)


@pytest.mark.parametrize("shift", [1, 2, 8])
def test_product_of_buffers_at_any_byte(shift):
    product("bf16", [[5, 70], [0, 3]], 80, 256, 136, shift)


def test_product_several_tiles_of_a_block():
    product("bf16", [[700, 500, 256], [0, 513, 31]], 1500, 1024, 4104)


def test_a_nan_stays_in_its_row_and_column():
    x8, w8 = torch.ones(1, 200, 256, device="cuda").to(F8), torch.ones(1, 1, 256, 256, device="cuda").to(F8)
    xs, ws = torch.ones(1, 200, 2, device="cuda"), torch.ones(1, 1, 2, 2, device="cuda")
    off = torch.tensor([[0, 200]], dtype=torch.int32, device="cuda")
    x8.view(torch.uint8)[0, 3, 0] = 0x7f
    w8.view(torch.uint8)[0, 0, 130, 200] = 0xff
    xs[0, 150, 1], ws[0, 0, 1, 0] = float("inf"), 2.0
    out = torch.empty(1, 200, 256, device="cuda")
    vc.vc_expert_product_fp8(x8, xs, w8, ws, off, out)
    want = torch.full((200, 256), 256.0, device="cuda")
    want[:, 128:] = 384
    want[150] = float("inf")
    want[3], want[:, 130] = float("nan"), float("nan")
    assert torch.equal(torch.nan_to_num(out[0], nan=-1), torch.nan_to_num(want, nan=-1))


def test_dispatched_replayed_and_again():
    """Tokens rounded on their ranks, dispatched with their scales, multiplied;
    the same bits from a graph."""
    N, rows, H, E, k, F = 4, 33, 384, 8, 2, 264
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(N, rows, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, E // N, F, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, E, (N, rows, k), generator=g, device="cuda", dtype=torch.int32)
    cap = N * rows * k
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    slots, off = torch.empty(N, rows, k, **i32), torch.empty(N, E // N + 1, **i32)
    x8, xs = torch.empty(N, rows, H, dtype=F8, device="cuda"), torch.empty(N, rows, blocks(H), **f32)
    w8, ws = torch.empty(w.shape, dtype=F8, device="cuda"), torch.empty(N, E // N, blocks(F), blocks(H), **f32)
    r8, rs = torch.zeros(N, cap, H, dtype=F8, device="cuda"), torch.zeros(N, cap, blocks(H), **f32)
    out = torch.zeros(N, cap, F, dtype=torch.bfloat16, device="cuda")
    vc.vc_quantize_fp8(w, w8, ws, block_rows=128)

    def go():
        vc.vc_quantize_fp8(x, x8, xs)
        vc.vc_dispatch_plan(ids, slots, off, cap)
        vc.vc_dispatch(x8, slots, r8)
        vc.vc_dispatch(xs, slots, rs)
        vc.vc_expert_product_fp8(r8, rs, w8, ws, off, out)
    go()
    torch.cuda.synchronize()
    want = out.clone()
    X, W = values(x8, xs, 1), values(w8, ws, 128)
    for r in range(N):
        for t in range(rows):
            for j in range(k):
                d, p = divmod(int(slots[r, t, j]), cap)
                e = int(ids[r, t, j])
                assert e // (E // N) == d
                a, b = X[r, t], W[d, e % (E // N)]
                bound = (H + 10) * ref.ULP * (np.abs(b) @ np.abs(a)) + store_bound(b @ a, "bf16")
                assert (np.abs(f64(out[d, p]) - b @ a) <= bound).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_rows_beyond_32_bits_of_elements():
    cap, win, width = 2 ** 20 + 100, 2048 + 128, 256
    first = cap - 64
    assert first * win > 2 ** 31
    x = torch.zeros(1, cap, win, dtype=torch.bfloat16, device="cuda")
    x[0, first:].copy_(torch.randn(64, win, device="cuda"))
    x8, xs = torch.empty(1, cap, win, dtype=F8, device="cuda"), torch.empty(1, cap, blocks(win), device="cuda")
    vc.vc_quantize_fp8(x, x8, xs)
    check_quantized([x[0, first:]], [x8[0, first:]], [xs[0, first:]], 1)
    assert bool((xs[0, :first] == 0).all())
    w = torch.randn(1, 1, width, win, device="cuda")
    w8, ws = torch.empty(1, 1, width, win, dtype=F8, device="cuda"), torch.empty(1, 1, blocks(width), blocks(win), device="cuda")
    vc.vc_quantize_fp8(w, w8, ws, block_rows=128)
    off = torch.tensor([[first, cap]], dtype=torch.int32, device="cuda")
    out = torch.full((1, cap, width), 7.0, device="cuda")
    vc.vc_expert_product_fp8(x8, xs, w8, ws, off, out)
    X, W = values(x8[0, first:], xs[0, first:], 1), values(w8[0], ws[0], 128)[0]
    bound = (win + 2 * blocks(win) + 2) * ref.ULP * (np.abs(X) @ np.abs(W).T) + store_bound(X @ W.T, "f32")
    assert (np.abs(f64(out[0, first:]) - X @ W.T) <= bound).all() and bool((out[0, :first] == 7).all())
