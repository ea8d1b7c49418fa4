"""The experts' products and their gradients against 64-bit products, within
bounds derived in tests/expert_ref.py: types, both layouts of the weights, odd
and whole widths, buffers at any element, and what the rows behind the last
expert's hold before and after."""
import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import expert_ref as ref
from .layer_ref import DT, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def made(*shape, dt, g, by=1.0, shift=0):
    """Normal numbers, each rank's buffer `shift` elements off a boundary."""
    n = int(np.prod(shape[1:], dtype=np.int64))
    out = []
    for _ in range(shape[0]):
        room = torch.zeros(n + shift + 64, dtype=DT[dt], device="cuda")
        t = room[shift:shift + n].view(shape[1:])
        t.copy_(torch.randn(*shape[1:], generator=g, device="cuda") * by)
        out.append(t)
    return out


def host(ts):
    return np.stack([f64(t) for t in ts])


def offsets_of(rows):
    ends = np.concatenate([np.zeros((len(rows), 1), np.int64), np.cumsum(rows, 1)], 1).astype(np.int32)
    return torch.from_numpy(ends).cuda()


def inputs(dt, rows, cap, win, width, transposed, shift=0, seed=0):
    N, each = np.asarray(rows).shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = made(N, cap, win, dt=dt, g=g, shift=shift)
    w = made(N, each, *((width, win) if transposed else (win, width)), dt=dt, g=g, by=max(win, 1) ** -0.5, shift=shift)
    dy = made(N, cap, width, dt=dt, g=g, shift=shift)
    return x, w, dy, offsets_of(rows)


def check(got, want, bound, what):
    assert np.isfinite(want).all()
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} want {want[bad][0]} +- {bound[bad][0]}"


def run(dt, rows, cap, win, width, transposed, shift=0, wide=False):
    x, w, dy, off = inputs(dt, rows, cap, win, width, transposed, shift)
    last = [int(e) for e in off[:, -1]]
    for d, n in enumerate(last):  # no expert's rows must not matter
        x[d][n:], dy[d][n:] = float("nan"), float("inf")
    out, dx = (made(len(x), cap, n, dt=dt, g=torch.Generator(device="cuda").manual_seed(9), shift=shift) for n in (width, win))
    dw = [torch.full(t.shape, float("nan"), dtype=torch.float32 if wide else t.dtype, device="cuda") for t in w]
    kept = host(out), host(dx)
    vc.vc_expert_product(x, w, off, out, transposed=transposed)
    vc.vc_expert_product_backward(dy, x, w, off, drows=dx, dweight=dw, transposed=transposed)
    torch.cuda.synchronize()
    X, W, dY = (host(t) for t in (x, w, dy))
    check(host(out), *ref.product(X, W, off.cpu(), kept[0], transposed, dt), "out")
    check(host(dx), *ref.product(dY, W, off.cpu(), kept[1], not transposed, dt), "drows")
    check(host(dw), *ref.weight_grad(dY, X, off.cpu(), W.shape, transposed, "f32" if wide else dt), "dweight")


ROWS = {
    "one": ([[1]], 1),
    "none": ([[0, 0], [0, 0]], 3),
    "few": ([[3, 0, 1, 2], [0, 0, 0, 5]], 9),
    "full": ([[64, 64]], 128),
    "ragged": ([[17, 130, 0], [1, 257, 33], [0, 0, 300]], 301),
    "long": ([[0, 1100], [513, 15]], 1100),
}
WIDTHS = [(64, 128), (512, 256), (8, 8), (128, 640), (200, 72), (1003, 515), (1, 1), (7, 300), (300, 7), (65, 129)]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", ROWS)
def test_rows(dt, transposed, rows):
    run(dt, *ROWS[rows], 136, 200, transposed)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("win,width", WIDTHS)
def test_widths(dt, transposed, win, width):
    run(dt, *ROWS["ragged"], win, width, transposed, wide=win % 2 == 1)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_buffers_at_any_element(dt, shift):
    run(dt, *ROWS["ragged"], 136, 72, False, shift=shift)
    run(dt, *ROWS["few"], 64, 66, True, shift=shift, wide=True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_several_tiles_of_a_block(dt, transposed):
    """More tiles than the GPU has multiprocessors, long sums, and experts
    whose pieces are longer than those of one with more rows."""
    run(dt, [[700, 500, 256], [0, 513, 31]], 1500, 648, 4104, transposed)


def test_many_ranks_and_experts():
    rng = np.random.RandomState(0)
    run("bf16", rng.randint(0, 9, (64, 16)), 130, 72, 40, True)
    run("f16", rng.randint(0, 3, (1, 1024)), 2048, 64, 136, False, wide=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_widths_of_nothing(dt):
    """A sum over nothing is 0; a gradient over no rows too."""
    x, w, dy, off = inputs(dt, [[2, 3]], 8, 0, 16, False)
    out = torch.full((1, 8, 16), 7.0, dtype=DT[dt], device="cuda")
    vc.vc_expert_product(x, w, off, out)
    assert (out[0, :5] == 0).all() and (out[0, 5:] == 7).all()
    dw = torch.full((1, 2, 8, 16), 7.0, dtype=DT[dt], device="cuda")
    none = torch.empty(1, 0, 16, dtype=DT[dt], device="cuda"), torch.empty(1, 0, 8, dtype=DT[dt], device="cuda")
    vc.vc_expert_product_backward(*none, None, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), dweight=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("ends", [[[-5, 4, 400]], [[3, 2, 6]], [[0, 300, 300]], [[2 ** 31 - 1, -2 ** 31, 5]]])
def test_offsets_outside_the_buffer(dt, ends):
    """Taken into [0, capacity], and an end before its beginning as none."""
    x, w, dy, _ = inputs(dt, [[4, 4]], 70, 64, 72, True)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 70, 72, dtype=DT[dt], device="cuda")
    dx, dw = torch.zeros(1, 70, 64, dtype=DT[dt], device="cuda"), torch.empty(1, 2, 72, 64, dtype=DT[dt], device="cuda")
    vc.vc_expert_product(x, w, off, out, transposed=True)
    vc.vc_expert_product_backward(dy, x, w, off, drows=dx, dweight=dw, transposed=True)
    X, W, dY = (host(t) for t in (x, w, dy))
    if ends != [[3, 2, 6]]:
        check(f64(out), *ref.product(X, W, off.cpu(), np.zeros(out.shape), True, dt), "out")
        check(f64(dx), *ref.product(dY, W, off.cpu(), np.zeros(dx.shape), False, dt), "drows")
    check(f64(dw), *ref.weight_grad(dY, X, off.cpu(), W.shape, True, dt), "dweight")


def test_infinities_and_nan_stay_in_their_rows():
    for dt in ("f32", "bf16"):
        x, w, dy, off = inputs(dt, [[40, 30]], 80, 72, 64, False)
        clean, out = (torch.zeros(1, 80, 64, dtype=DT[dt], device="cuda") for _ in range(2))
        vc.vc_expert_product(x, w, off, clean)
        x[0][3, 5], x[0][45, 0] = float("inf"), float("nan")
        vc.vc_expert_product(x, w, off, out)
        bad = ~torch.isfinite(out[0]).all(1)
        assert bad.nonzero()[:, 0].tolist() == [3, 45]
        keep = ~bad
        assert torch.equal(out[0][keep], clean[0][keep])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("win,width", [(72, 136), (71, 137)])
def test_weights_of_experts_without_rows_do_not_matter(dt, win, width):
    x, w, dy, off = inputs(dt, [[5, 0, 40], [0, 20, 0]], 50, win, width, False)
    w[0][1], w[1][0], w[1][2] = float("nan"), float("inf"), float("nan")
    out, dx = (torch.zeros(2, 50, n, dtype=DT[dt], device="cuda") for n in (width, win))
    vc.vc_expert_product(x, w, off, out)
    vc.vc_expert_product_backward(dy, None, w, off, drows=dx)
    w[0][1], w[1][0], w[1][2] = 0, 0, 0
    X, W, dY = (host(t) for t in (x, w, dy))
    check(f64(out), *ref.product(X, W, off.cpu(), np.zeros(out.shape), False, dt), "out")
    check(f64(dx), *ref.product(dY, W, off.cpu(), np.zeros(dx.shape), True, dt), "drows")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_beyond_32_bits_of_elements(dt):
    """The rows stand behind the first 2^31 elements of their buffers."""
    cap, win, width = 2 ** 20 + 300, 2048 + 8, 2048 + 16
    first = cap - 200
    assert first * win > 2 ** 31
    x, dy = (torch.zeros(1, cap, n, dtype=DT[dt], device="cuda") for n in (win, width))
    g = torch.Generator(device="cuda").manual_seed(0)
    x[0, first:].copy_(torch.randn(200, win, generator=g, device="cuda"))
    dy[0, first:].copy_(torch.randn(200, width, generator=g, device="cuda"))
    w = (torch.randn(1, 2, win, width, generator=g, device="cuda") * win ** -0.5).to(DT[dt])
    off = torch.tensor([[first, first + 130, cap]], dtype=torch.int32, device="cuda")
    out, dx = torch.full_like(dy, 7), torch.full_like(x, 7)
    dw = torch.empty_like(w)
    vc.vc_expert_product(x, w, off, out)
    vc.vc_expert_product_backward(dy, x, w, off, drows=dx, dweight=dw)
    tail = torch.tensor([[0, 130, 200]])
    X, W, dY = (np.stack([f64(t)]) for t in (x[0, first:], w[0], dy[0, first:]))
    check(f64(out[:, first:]), *ref.product(X, W, tail, np.zeros((1, 200, width)), False, dt), "out")
    check(f64(dx[:, first:]), *ref.product(dY, W, tail, np.zeros((1, 200, win)), True, dt), "drows")
    check(f64(dw), *ref.weight_grad(dY, X, tail, W.shape, False, dt), "dweight")
    assert bool((out[0, :first] == 7).all()) and bool((dx[0, :first] == 7).all())


def test_two_threads_on_two_streams():
    """Calls of two host threads on streams of their own, 16-bit and 8-bit
    products at once, give the bits of calls by themselves."""
    import threading
    x, w, dy, off = inputs("bf16", [[100, 300], [0, 77]], 400, 264, 384, False)
    odd = inputs("f16", [[30, 9], [60, 1]], 100, 131, 77, True, seed=3)
    f8 = [torch.randn(2, 400, 256, device="cuda").to(torch.float8_e4m3fn), torch.rand(2, 400, 2, device="cuda"),
          torch.randn(2, 2, 384, 256, device="cuda").to(torch.float8_e4m3fn), torch.rand(2, 2, 3, 2, device="cuda"), off]

    def buffers():
        return [torch.zeros(2, 400, 384, dtype=DT["bf16"], device="cuda"), torch.zeros(2, 2, 264, 384, dtype=DT["bf16"], device="cuda"),
                torch.zeros(2, 100, 77, dtype=DT["f16"], device="cuda"), torch.zeros(2, 400, 384, device="cuda")]

    def go(b, stream=None):
        vc.vc_expert_product(x, w, off, b[0], stream=stream)
        vc.vc_expert_product_fp8(*f8, b[3], stream=stream)
        vc.vc_expert_product_backward(dy, x, w, off, dweight=b[1], stream=stream)
        vc.vc_expert_product(odd[0], odd[1], odd[3], b[2], transposed=True, stream=stream)
    want = buffers()
    go(want)
    torch.cuda.synchronize()
    got, failed = [buffers() for _ in range(2)], []

    def many(b, stream):
        try:
            for _ in range(300):
                go(b, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=many, args=(b, torch.cuda.Stream())) for b in got]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and vc.vc_device_errors() == 0
    for b in got:
        assert all(torch.equal(a, c) for a, c in zip(b, want))


def test_same_bits_again_and_on_another_stream_and_replayed():
    x, w, dy, off = inputs("bf16", [[100, 300], [0, 77]], 400, 256, 384, True)
    out, dx, dw = torch.zeros(2, 400, 384, dtype=DT["bf16"], device="cuda"), torch.zeros(2, 400, 256, dtype=DT["bf16"], device="cuda"), \
        torch.zeros(2, 2, 384, 256, dtype=DT["bf16"], device="cuda")

    def go(stream=None):
        vc.vc_expert_product(x, w, off, out, transposed=True, stream=stream)
        vc.vc_expert_product_backward(dy, x, w, off, drows=dx, dweight=dw, transposed=True, stream=stream)
    go()
    want = [t.clone() for t in (out, dx, dw)]

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, dx, dw), want))
        for t in (out, dx, dw):
            t.zero_()
        torch.cuda.synchronize()
    same()
    side = torch.cuda.Stream()
    go(side)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        graph.replay()
        same()
    assert vc.vc_device_errors() == 0


def test_pairs_of_blocks_behind_a_kernel_that_leaves_one_by_one():
    """Many passes enqueued ahead, weights copied to 16-byte boundaries before
    each product: a pair's blocks start apart, and meet before they share tensor
    memory."""
    g = torch.Generator(device="cuda").manual_seed(0)
    N, each, cap, win, width = 8, 5, 32, 1089, 2473
    x, w = made(N, cap, win, dt="bf16", g=g), made(N, each, win, width, dt="bf16", g=g)
    offs = [offsets_of(torch.randint(0, 3, (N, each), generator=torch.Generator().manual_seed(k)).numpy()) for k in range(3)]
    outs = [torch.zeros(N, cap, width, dtype=DT["bf16"], device="cuda") for _ in range(3)]
    for i in range(3):
        vc.vc_expert_product(x, w, offs[i], outs[i])
    want = [t.clone() for t in outs]
    for _ in range(20):
        for j in range(600):
            vc.vc_expert_product(x, w, offs[j % 3], outs[j % 3])
        assert vc.vc_device_errors() == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
