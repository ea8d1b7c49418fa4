"""vc_route and its backward on the GPU against the definition in 64 bits.

Choices are compared exactly.  Where experts are compared by the logits
themselves that needs no margin; where by scores, a token counts only if what
decides is 1e-5 of its size apart: a score is exp (2 roundings, and the error
of its argument, at most 15 here, times u), a sum of ten levels and a
division, so within 32 u = 2e-6, and a group's or a biased score adds two
roundings more.  Most tokens count (checked).
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


def run(logits, topk, **how):
    N, rows, E = logits.shape
    ids = torch.full((N, rows, topk), -7, dtype=torch.int32, device="cuda")
    w = torch.full((N, rows, topk), -7.0, device="cuda")
    vc.vc_route(logits, ids, w, **how)
    return ids.cpu().numpy(), ref.f64(w)


def check(logits, bias, score, topk, ngroups=1, keep=1, top=1, renorm=True, scale=1.0, margin=True):
    how = dict(score=score, ngroups=ngroups, topk_groups=keep, group_top=top, renormalize=renorm, scale=scale)
    ids, w = run(logits, topk, bias=bias, **how)
    l64 = ref.f64(logits)
    b64 = None if bias is None else ref.f64(bias)
    by_score = bias is not None or (ngroups > 1 and top == 2)
    N, rows, _ = l64.shape
    counted = 0
    for r in range(N):
        for t in range(rows):
            want, ww, gap = ref.route_row(l64[r, t], None if b64 is None else (b64[r] if b64.ndim == 2 else b64), score,
                                          topk, ngroups, keep, top, renorm, scale)
            if by_score and margin and gap < 1e-5:
                continue
            counted += 1
            assert np.array_equal(ids[r, t], want), (r, t, ids[r, t], want, gap)
            # exp and the division round a few times; exp's argument error is |l - max| u
            span = np.ptp(l64[r, t][np.isfinite(l64[r, t])]) if np.isfinite(l64[r, t]).any() else 0
            assert np.all(np.abs(w[r, t] - ww) <= (2 * span + 60) * ref.U32 * np.abs(ww) + 1e-37), (r, t, w[r, t], ww)
    assert counted > N * rows // 2


SHAPES = [  # E, topk, ngroups, keep: one expert, odd counts, a group of a lane's part, of lanes, of odd parts
    (1, 1, 1, 1), (2, 2, 1, 1), (7, 3, 1, 1), (32, 4, 8, 2), (33, 5, 3, 2), (60, 6, 4, 2), (64, 8, 8, 3),
    (96, 8, 32, 7), (128, 32, 1, 1), (160, 6, 8, 3), (256, 8, 8, 4), (384, 8, 2, 1), (512, 8, 16, 4), (1000, 10, 5, 2),
    (1024, 16, 32, 8),
]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,topk,G,keep", SHAPES)
def test_choices(E, topk, G, keep, dt):
    g = torch.Generator().manual_seed(E)
    logits = (torch.randn(2, 9, E, generator=g) * 1.5).to(ref.DT[dt]).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda()
    for score in ("softmax", "sigmoid"):
        check(logits, None, score, topk, renorm=True, scale=2.5)
        check(logits, None, score, topk, G, keep, 1, renorm=False)
        check(logits, None, score, topk, G, keep, 2)
        check(logits, bias, score, topk, renorm=False)
        check(logits, bias, score, topk, G, keep, 2, scale=0.5)
        check(logits, torch.stack([bias, -bias]), score, topk, G, keep, 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 60, 256])
def test_ties_go_to_the_lower_index(score, E):
    logits = torch.zeros(1, 3, E)
    logits[0, 1, E // 2:] = 1.0
    logits[0, 2, ::2] = -0.0
    logits = logits.cuda()
    zero = torch.zeros(E, device="cuda")
    for bias in (None, zero):
        check(logits, bias, score, 4, margin=False)
        check(logits, bias, score, 4, 4, 2, 1, margin=False)
        check(logits, bias, score, 4, 4, 2, 2, margin=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(24, 4), (256, 8)])
def test_masks(score, E, G):
    """-inf, NaN, +inf and the lowest finite logits; rows with too few experts, or none."""
    x = torch.randn(1, 8, E)
    x[0, 0] = -float("inf")
    x[0, 1] = -float("inf")
    x[0, 1, 5] = 0.25
    x[0, 2] = torch.finfo(torch.float32).min
    x[0, 3] = torch.finfo(torch.float32).min
    x[0, 3, 9] = 1.0
    x[0, 4] = float("nan")
    x[0, 5, ::2] = float("nan")
    x[0, 6, 3] = float("inf")
    x[0, 7, : E - 3] = -float("inf")
    x = x.cuda()
    bias = (torch.arange(E) % 7).float().cuda() * 0.0625
    for b in (None, bias):
        for renorm in (True, False):
            check(x, b, score, 6, renorm=renorm, margin=False)
            check(x, b, score, 6, G, 2, 1, renorm=renorm, margin=False)
    ids, w = run(x, 6, score=score)
    assert (ids[0, 0] == -1).all() and (w[0, 0] == 0).all()
    assert ids[0, 1].tolist() == [5, -1, -1, -1, -1, -1] and w[0, 1, 0] == 1
    assert (ids[0, 4] == -1).all() and (w[0, 4] == 0).all()
    blocked = torch.full((E,), -float("inf"), device="cuda")
    blocked[3] = 0
    ids, w = run(x[:, 7:], 2, score=score, bias=blocked)
    assert (ids == -1).all() and (w == 0).all()


def test_scores_are_elementary_fp32_operations():
    """Scores plus bias choose as single fp32 operations do, bit for bit: equal
    bf16 logits are common, and biases of a few roundings decide among them."""
    g = torch.Generator().manual_seed(0)
    l = torch.randn(1, 4096, 64, generator=g).to(torch.bfloat16).cuda()
    bias = (torch.randn(64, generator=g) * 1e-6).cuda()
    ids, _ = run(l, 8, score="sigmoid", bias=bias)
    x = l.float()
    c = 1 / (1 + torch.exp(-x)) + bias
    want = torch.sort(c, dim=-1, descending=True, stable=True)[1][..., :8]
    assert np.array_equal(ids, want.cpu().numpy())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,topk", [(1, 1), (7, 3), (33, 5), (128, 6), (256, 8), (1000, 32)])
def test_backward(E, topk, dt):
    N, rows, scale = 2, 5, 1.75
    g = torch.Generator().manual_seed(E + 1)
    logits = torch.randn(N, rows, E, generator=g).to(ref.DT[dt]).cuda()
    logits[1, 4] = -float("inf")
    dw = torch.randn(N, rows, topk, generator=g).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = torch.empty(N, rows, topk, dtype=torch.int32, device="cuda"), torch.empty(N, rows, topk, device="cuda")
            vc.vc_route(logits, ids, w, score=score, renormalize=renorm, scale=scale)
            if topk > 2:
                ids[0, 0, 1] = -1       # takes no part
                ids[0, 1, 2] = E + 5    # neither does this
            dl = torch.full_like(logits, 7)
            vc.vc_route_backward(dw, logits, ids, dl, score=score, renormalize=renorm, scale=scale)
            got, l64, d64, id64 = ref.f64(dl), ref.f64(logits), ref.f64(dw), ids.cpu().numpy()
            for r in range(N):
                for t in range(rows):
                    l, i = l64[r, t], np.where(id64[r, t] < E, id64[r, t], -1)
                    s, _ = ref.scores(l, score)
                    p = np.where(i >= 0, s[np.maximum(i, 0)], 0.0)
                    d = np.where(i >= 0, d64[r, t] * scale, 0.0)
                    S = p.sum() if renorm else 1.0
                    ds, mag = np.zeros(E), np.zeros(E)
                    dot = (d * p).sum() / S if renorm and S else 0.0
                    for j in range(topk):
                        if i[j] >= 0 and S:
                            ds[i[j]] += (d[j] - dot) / S
                            mag[i[j]] += (np.abs(d[j]) + np.abs(d * p).sum() / S) / S
                    if score == "sigmoid":
                        want, size = ds * s * (1 - s), mag * s
                    else:
                        rest = 0.0 if renorm else (ds * s).sum()
                        want, size = s * (ds - rest), s * (mag + (0 if renorm else (mag * s).sum()))
                    # up to topk + 20 roundings of terms of these magnitudes, and exp's argument error
                    span = np.ptp(l[np.isfinite(l)]) if np.isfinite(l).any() else 0
                    bound = (topk + 40 + 4 * span) * ref.U32 * size + ref.store_bound(want, dt) + 1e-37
                    assert np.all(np.abs(got[r, t] - want) <= bound), (score, renorm, r, t, np.abs(got[r, t] - want).max())


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_backward_against_differences(score, renorm):
    """Central differences of the 64-bit weights of fixed choices: truncation
    of order e^2 = 1e-10, under the fp32 gradient's 1e-6 of the magnitudes."""
    E, topk = 20, 4
    logits = torch.randn(1, 6, E).cuda()
    ids, w = torch.empty(1, 6, topk, dtype=torch.int32, device="cuda"), torch.empty(1, 6, topk, device="cuda")
    vc.vc_route(logits, ids, w, score=score, renormalize=renorm)
    dw, dl = torch.randn(1, 6, topk).cuda(), torch.empty_like(logits)
    vc.vc_route_backward(dw, logits, ids, dl, score=score, renormalize=renorm)
    l64, d64, id64, got = ref.f64(logits)[0], ref.f64(dw)[0], ids.cpu().numpy()[0], ref.f64(dl)[0]
    e = 1e-5
    for t in range(6):
        for i in range(E):
            up, down = l64[t].copy(), l64[t].copy()
            up[i] += e
            down[i] -= e
            slope = ((ref.route_weights(up, id64[t], score, renorm, 1.0) -
                      ref.route_weights(down, id64[t], score, renorm, 1.0)) * d64[t]).sum() / (2 * e)
            assert abs(slope - got[t, i]) <= 2e-6 * np.abs(d64[t]).sum(), (t, i)


def test_unaligned_rows_and_another_stream():
    raw = torch.randn(3 * 64 + 1).to(torch.bfloat16).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = []
    for x in (raw[1:].view(1, 3, 64), raw[1:].clone().view(1, 3, 64)):
        ids, w = torch.empty(1, 3, 4, dtype=torch.int32, device="cuda"), torch.empty(1, 3, 4, device="cuda")
        vc.vc_route(x, ids, w, stream=s)
        dl = torch.empty(193, dtype=torch.bfloat16, device="cuda")[1 if not out else 0:][:192].view(1, 3, 64)
        vc.vc_route_backward(w, x, ids, dl, renormalize=False, stream=s)
        out.append((ids, w, dl))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_no_tokens():
    e = torch.empty(2, 0, 8, device="cuda")
    ids, w = torch.empty(2, 0, 2, dtype=torch.int32, device="cuda"), torch.empty(2, 0, 2, device="cuda")
    vc.vc_route(e, ids, w)
    vc.vc_route_backward(w, e, ids, torch.empty_like(e))
