"""vc_route and its backward at the ends of the number range, against the
definition in 64 bits, and its choices bit for bit."""
import numpy as np
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from . import layer_ref as ref
from .test_gpu_route import check

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126  # the smallest sum of chosen scores that weights are divided by


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def far(E, best, below, at):
    """Logits whose largest is `best`, at the expert after the chosen ones at
    `at`, which lie `below` it and a little more; the rest between."""
    l = torch.linspace(best - 3, best - 40, E)
    l[at + 3] = best
    l[at:at + 3] = best - below - torch.tensor([0.0, 1.0, 2.5])
    return l


ROWS = [  # largest logit, how far below it the chosen ones lie; the sum of their scores over 2^-126 = exp(-87.3)
    (0.0, 100.0),   # far under
    (200.0, 200.0), # far under, of large logits
    (3.0, 130.0),   # under fp32's smallest subnormal
    (0.0, 84.0),    # over, within a few thousand rows' softmax sums of it for few experts
    (0.0, 60.0),    # over
    (0.0, 1.0),     # ordinary
    (-5.0, 60.0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,at", [(7, 0), (40, 30), (100, 41), (256, 250), (1000, 500)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_of_vanishing_scores(score, E, at, dt):
    """A bias chooses experts whose scores sum to less than 2^-126, or to just
    more.  Below, the gradient is 0 (the weights are not shares of the sum
    there); above, the shares' gradient.  Bounds as in test_gpu_route's
    backward: up to topk + 20 roundings of terms of these magnitudes, twice,
    and the error of exp's argument (differences of logits here)."""
    topk, scale = 3, 1.75
    logits = torch.stack([far(E, *row, at) for row in ROWS])[None].to(ref.DT[dt]).cuda()
    bias = torch.zeros(E, device="cuda")
    bias[at:at + 3] = torch.tensor([64.0, 32.0, 16.0])  # the order whatever the scores
    rows = len(ROWS)
    ids, w = torch.empty(1, rows, topk, dtype=torch.int32, device="cuda"), torch.empty(1, rows, topk, device="cuda")
    vc.vc_route(logits, ids, w, bias=bias, score=score, renormalize=True, scale=scale)
    assert (ids.cpu() == torch.tensor([at, at + 1, at + 2])).all()
    dw = torch.tensor([1.0, -1.0, 0.375]).repeat(1, rows, 1).cuda()
    dl = torch.full_like(logits, 7)
    vc.vc_route_backward(dw, logits, ids, dl, score=score, renormalize=True, scale=scale)
    l64, got, w64, d = ref.f64(logits)[0], ref.f64(dl)[0], ref.f64(w)[0], ref.f64(dw)[0, 0] * scale
    under = 0
    for t in range(rows):
        s = ref.scores(l64[t], score)[0][at:at + 3]
        total = s.sum()
        assert not 0.5 < total / LEAST < 2, "too near the limit to tell"
        want = np.zeros(E)
        size = np.zeros(E)
        if total >= LEAST:
            p = s / total
            grow = 1 - s if score == "sigmoid" else 1.0
            want[at:at + 3] = p * (d - (d * p).sum()) * grow
            size[at:at + 3] = p * (np.abs(d) + np.abs(d * p).sum())
        under += total < LEAST
        span = 40  # of the chosen logits' part in exp's argument, twice
        bound = (topk + 40 + 4 * span) * ref.U32 * size + ref.store_bound(want, dt) + 1e-37
        assert np.all(np.abs(got[t] - want) <= bound), (ROWS[t], total, got[t, at:at + 3], want[at:at + 3])
        # the forward's weights: shares of the larger of the sum and 2^-126 (softmax scores under it are subnormal in
        # fp32; a sigmoid's are 0 where exp(-logit) passes fp32's largest number)
        if score == "softmax":
            by = max(total, LEAST)
            off = np.abs(w64[t] - scale * s / by)
            assert np.all(off <= 1e-4 * scale * s / by + scale * 2.0 ** -148 / by), (ROWS[t], w64[t], scale * s / by)
    assert 2 <= under <= 4


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward_beside_infinite_and_absent_logits(dt):
    """+inf is the whole softmax, so choices beside it have no gradient, and
    where it is chosen itself the others' shares are 0; -inf and NaN are not
    there, chosen or not."""
    inf, nan = float("inf"), float("nan")
    logits = torch.tensor([[0.0, 1.0, inf, 2.0], [0.0, 1.0, inf, 2.0], [nan, 1.0, -inf, 2.0], [-inf, -inf, -inf, -inf],
                           [0.0, -inf, 500.0, -inf]])[None].to(ref.DT[dt]).cuda()
    ids = torch.tensor([[0, 3], [2, 3], [1, 3], [0, 1], [1, 3]], dtype=torch.int32)[None].cuda()
    dw, dl = torch.tensor([1.0, -1.0]).repeat(1, 5, 1).cuda(), torch.full_like(logits, 7)
    vc.vc_route_backward(dw, logits, ids, dl, score="softmax", renormalize=True)
    got = ref.f64(dl)[0]
    for t in (0, 1, 3, 4):
        assert not got[t].any(), (t, got[t])
    p = 1 / (1 + np.exp(1.0))  # the share of logit 1 against 2
    want = 2 * p * (1 - p)
    assert np.allclose(got[2], [0, want, 0, -want], rtol=2e-6 if dt == "f32" else 2.0 ** -8, atol=0)


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(8, 4), (24, 4), (64, 16), (128, 32), (256, 16), (160, 5), (1024, 32)])
def test_groups_biased_to_the_lowest_number(score, E, G):
    """A mask by the lowest finite bias: two such scores add up to less than
    any fp32 number, and yet their group has experts.  Kept groups, more than
    hold an ordinary expert, are then the lowest of the masked ones, which
    come before groups that a bias of -inf empties."""
    each = E // G
    logits = torch.randn(1, 4, E, generator=torch.Generator().manual_seed(E)).cuda()
    topk = min(32, 2 * each + 1)
    masked = torch.full((E,), LOWEST, device="cuda")
    for ordinary in ([], [1], [G - 1]):
        for empty in ([], [0], [0, 2]):
            bias = masked.clone()
            for g in empty:
                bias[g * each:(g + 1) * each] = -float("inf")
            for g in ordinary:
                bias[g * each:(g + 1) * each] = 0
            for keep in (1, 2, 3, G):
                for top in (1, 2):
                    check(logits, bias, score, topk, G, keep, top, margin=False)


def pairs(x):
    """The sum over the last dimension, neighbours first."""
    return x if x.shape[-1] == 1 else pairs(x[..., 0::2] + x[..., 1::2])


def scores32(l, score):
    """Scores as single fp32 operations in the documented order."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(-1, keepdim=True))
    pad = 2 ** (l.shape[-1] - 1).bit_length() - l.shape[-1]
    return e / pairs(torch.nn.functional.pad(e, (0, pad)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep", [(48, 1, 1), (60, 4, 2), (64, 8, 3), (200, 5, 2), (256, 8, 4), (1000, 1, 1), (1024, 32, 5)])
def test_choices_bit_for_bit(score, E, G, keep):
    """The order of experts and groups is that of the documented fp32
    operations, bit for bit: bf16 logits give many equal scores, and biases of
    a few roundings decide among them.  No token is left out."""
    rows, topk = 2048, 8
    g = torch.Generator().manual_seed(E + G)
    logits = torch.randn(1, rows, E, generator=g).to(torch.bfloat16).cuda()
    s = scores32(logits.float(), score)
    tiny = (torch.randn(E, generator=g) * 1e-6).cuda() * float(s.mean())
    for bias in (tiny, None) if G > 1 else (tiny,):
        ids = torch.empty(1, rows, topk, dtype=torch.int32, device="cuda")
        w = torch.empty(1, rows, topk, device="cuda")
        vc.vc_route(logits, ids, w, bias=bias, score=score, ngroups=G, topk_groups=keep, group_top=2)
        c = s if bias is None else s + bias
        if G > 1:
            best = torch.sort(c.view(1, rows, G, E // G), dim=-1, descending=True)[0]
            kept = torch.sort(best[..., 0] + best[..., 1], dim=-1, descending=True, stable=True)[1][..., :keep]
            on = torch.zeros(1, rows, G, dtype=torch.bool, device="cuda").scatter(-1, kept, True)
            c = torch.where(on.repeat_interleave(E // G, -1), c, -float("inf"))
        want = torch.sort(c, dim=-1, descending=True, stable=True)[1][..., :topk]
        assert torch.equal(ids.long(), want)
