"""Cases of the layer operators that stand next to the collectives: the norm at
a tensor-parallel layer's boundary, routing to experts, and the exchange of
tokens between the ranks that hold them and the ranks that hold the experts.

Each case names an operator ("op") and its sizes.  With ``own`` false, run()
computes it in elementary torch operations in fp32; with ``own`` true it calls
the library.  Every rank's buffers are slices of one tensor whose first
dimension is the virtual ranks.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
TINY = 2.0 ** -126  # the smallest sum of scores that weights are divided by


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One new token per rank during generation, eight tensor-parallel
        # partial sums each, quantised for an 8-bit product: latency.
        {"name": "norm-decode-i8", "op": "norm", "N": 8, "rows": 1, "H": 4096, "dt": "bf16", "i8": True},
        # A prompt of 2048 tokens split over eight ranks, wide model: bandwidth.
        {"name": "norm-prefill-i8", "op": "norm", "N": 8, "rows": 256, "H": 8192, "dt": "bf16", "i8": True},
        # Odd sizes, three ranks, output in the data type (a training forward).
        {"name": "norm-odd-f16", "op": "norm", "N": 3, "rows": 333, "H": 2045, "dt": "f16", "i8": False},
        # Backward of the norm over a training micro-batch, four ranks: the
        # gradient of every rank's partial sums, of the residual, of the weight.
        {"name": "norm-backward", "op": "norm_bwd", "N": 4, "rows": 1024, "H": 4096, "dt": "bf16"},
        # Routing of one token per rank during generation: latency.
        {"name": "route-decode", "op": "route", "N": 8, "rows": 1, "E": 64, "k": 4, "dt": "f32", "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "top": 1, "renorm": True},
        # Many experts in groups, sigmoid scores with a balance bias, a large
        # batch over eight ranks.
        {"name": "route-groups-bias", "op": "route", "N": 8, "rows": 2048, "E": 256, "k": 8, "dt": "bf16",
         "score": "sigmoid", "bias": True, "groups": 8, "keep": 4, "top": 2, "renorm": True},
        # Backward of softmax routing whose weights are not renormalised: the
        # gradient reaches every expert's logit.
        {"name": "route-backward", "op": "route_bwd", "N": 4, "rows": 4096, "E": 128, "k": 6, "dt": "f32",
         "score": "softmax", "renorm": False},
        # 8-bit tokens with their scales to the experts, a few tokens per rank.
        {"name": "dispatch-decode-i8", "op": "dispatch", "N": 8, "rows": 4, "H": 4096, "E": 64, "k": 4, "dt": "i8"},
        # A prompt's tokens to their experts: bandwidth.
        {"name": "dispatch-prefill", "op": "dispatch", "N": 8, "rows": 512, "H": 4096, "E": 64, "k": 8, "dt": "bf16"},
        # The experts' answers back, weighted and summed: bandwidth.
        {"name": "combine-prefill", "op": "combine", "N": 8, "rows": 512, "H": 4096, "E": 64, "k": 8, "dt": "bf16"},
        # Odd row length and rank count (rows start off 16-byte boundaries).
        {"name": "combine-odd-f16", "op": "combine", "N": 5, "rows": 77, "H": 1003, "E": 20, "k": 3, "dt": "f16"},
        # Backward of the weighted sum in a training step.
        {"name": "combine-backward", "op": "combine_bwd", "N": 4, "rows": 512, "H": 2048, "E": 32, "k": 4,
         "dt": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _fit(case, most):
    """`case` with fewer rows where it would cost more than `most` bytes."""
    while work(case)["bytes"] > most and case["rows"] > 1:
        case["rows"] = max(1, case["rows"] // 2)
    return case


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "route", "route", "route_bwd", "dispatch", "dispatch", "combine",
                     "combine", "combine_bwd"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    N = rng.choice([1, 2, 3, 4, 6, 8])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = _log(rng, 64, 8192)
    H = rng.choice([H, max(64, H // 8 * 8), max(64, H // 64 * 64), max(64, H // 64 * 64)])
    if H == 3 * 1024:
        H += 64
    rows = _log(rng, 1, 2048)
    if op == "norm":
        i8 = dt != "f32" and rng.random() < 0.5
        return _fit({"op": op, "N": N, "rows": rows, "H": H, "dt": dt, "i8": i8}, most)
    if op == "norm_bwd":
        return _fit({"op": op, "N": N, "rows": rows, "H": H, "dt": dt}, most)
    groups = rng.choice([1, 1, 2, 4, 8])
    E = N * groups * _log(rng, 1, max(1, 256 // (N * groups)))
    E = E if E > 1 else 8 * N
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    if op == "route":
        keep = rng.randint(1, groups)
        k = min(k, E // groups * keep)
        return _fit({"op": op, "N": N, "rows": rows, "E": E, "k": k, "dt": dt, "score": rng.choice(["softmax", "sigmoid"]),
                     "bias": rng.random() < 0.5, "groups": groups, "keep": keep, "top": rng.choice([1, 2]),
                     "renorm": rng.random() < 0.7}, most)
    if op == "route_bwd":
        return _fit({"op": op, "N": N, "rows": rows, "E": E, "k": k, "dt": dt, "score": rng.choice(["softmax", "sigmoid"]),
                     "renorm": k > 1 and rng.random() < 0.5}, most)  # one renormalised weight is constant
    if op == "dispatch" and rng.random() < 0.4:
        dt = "i8"
    return _fit({"op": op, "N": N, "rows": rows, "H": H, "E": E, "k": k, "dt": dt}, most)


def _size(dt):
    return {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}[dt]


def work(case):
    c, op = case, case["op"]
    T, es = c["N"] * c["rows"], _size(c["dt"])
    if op == "norm":  # partial sums, residual, weight in; residual, output, scale and 1/rms out
        n, H = c["N"], c["H"]
        byts = T * H * es * (n + 2) + H * es + T * H * (1 if c["i8"] else es) + T * 4 * (2 if c["i8"] else 1)
        return {"bytes": byts, "flops": T * H * (n + (9 if c["i8"] else 5))}
    if op == "norm_bwd":  # two gradients, h, 1/rms, weight in; N copies of the gradient, the residual's, the weight's out
        n, H = c["N"], c["H"]
        return {"bytes": T * H * es * (3 + n + 1) + T * 4 + H * es + n * H * 4, "flops": T * H * 12}
    if op == "route":
        E, k = c["E"], c["k"]
        return {"bytes": T * E * es + T * k * 8 + (E * 4 if c["bias"] else 0), "flops": T * E * 6}
    if op == "route_bwd":  # with renormalised weights or sigmoid scores only the chosen logits are read
        E, k = c["E"], c["k"]
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * E * es + T * (E if dense else k) * es + T * k * 8, "flops": T * (E * 6 if dense else k * 10)}
    H, k = c["H"], c["k"]
    if op == "dispatch":  # ids in, slots and offsets out; each row in once and out k times, 8-bit rows with a scale
        row = H * es + (4 if c["dt"] == "i8" else 0)
        return {"bytes": T * row * (1 + k) + T * k * 8 + (c["E"] + c["N"]) * 4, "flops": T * k}
    if op == "combine":
        return {"bytes": T * H * es * (1 + k) + T * k * 8, "flops": T * k * H * 2}
    return {"bytes": T * H * es * (1 + 2 * k) + T * k * 12, "flops": T * k * H * 3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _capacity(c):
    """Rows a rank has room for: every row it could be sent where that is
    little, else a quarter above the mean (what goes over it is dropped)."""
    most = c["N"] * c["rows"] * min(c["k"], c["E"] // c["N"])
    return min(most, max(256, -(-5 * c["rows"] * c["k"] // 4)))


def _ids(c, g):
    """Distinct experts for each token, some experts more popular than others;
    the last rows of the last rank are padding (-1)."""
    N, rows, E, k = c["N"], c["rows"], c["E"], c["k"]
    liking = torch.randn(E, generator=g, device="cuda") * 0.3
    noise = -torch.log(-torch.log(torch.rand(N, rows, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    ids = torch.sort(liking + noise, dim=-1, descending=True, stable=True)[1][..., :k].to(torch.int32)
    ids[-1, rows - rows // 16:] = -1
    return ids.contiguous()


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dt=None, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(dt or DT[c["dt"]])

    def room(*shape, dt=None):
        return torch.zeros(*shape, dtype=dt or DT[c["dt"]], device="cuda")

    N, rows = c["N"], c["rows"]
    s = {"c": c}
    if op == "norm":
        H = c["H"]
        s["send"] = normal(N, N * rows, H, by=1 / math.sqrt(N))
        s["residual"] = normal(N, rows, H, by=2.0)
        s["weight"] = (1 + torch.randn(H, generator=g, device="cuda") * 0.1).to(DT[c["dt"]])
        s["residual_out"], s["rstd"] = room(N, rows, H), room(N, rows, dt=torch.float32)
        if c["i8"]:
            s["out"], s["scale"] = room(N, rows, H, dt=torch.int8), room(N, rows, dt=torch.float32)
            s["value"] = room(N, rows, H)
        else:
            s["out"] = room(N, rows, H)
    elif op == "norm_bwd":
        H = c["H"]
        s["dout"], s["dresidual_out"] = normal(N, rows, H), normal(N, rows, H)
        s["h"] = normal(N, rows, H, by=2.0)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
        s["weight"] = (1 + torch.randn(H, generator=g, device="cuda") * 0.1).to(DT[c["dt"]])
        s["dsend"], s["dresidual"] = room(N, N * rows, H), room(N, rows, H)
        s["dweight"] = room(N, H, dt=torch.float32)
    elif op in ("route", "route_bwd"):
        E, k = c["E"], c["k"]
        s["logits"] = normal(N, rows, E, by=1.5)
        s["logits"][-1, rows - rows // 16:] = -math.inf  # padding at the end of the last rank's rows
        if op == "route":
            s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if c["bias"] else None
            s["ids"], s["weights"] = room(N, rows, k, dt=torch.int32), room(N, rows, k, dt=torch.float32)
        else:
            top, ids = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
            s["ids"] = torch.where(top > -math.inf, ids, -1)[..., :k].to(torch.int32).contiguous()
            s["dweights"] = normal(N, rows, k, dt=torch.float32)
            s["dlogits"] = room(N, rows, E)
    else:
        H, E, k, cap = c["H"], c["E"], c["k"], _capacity(c)
        ids = _ids(c, g)
        if op == "dispatch":
            s["ids"], s["capacity"] = ids, cap
            if c["dt"] == "i8":
                s["send"] = torch.randint(-127, 128, (N, rows, H), generator=g, device="cuda", dtype=torch.int8)
                s["scale"] = torch.rand(N, rows, generator=g, device="cuda") * 0.05
                s["recv"], s["recv_scale"] = room(N, cap, H, dt=torch.int8), room(N, cap, dt=torch.float32)
            else:
                s["send"], s["recv"] = normal(N, rows, H), room(N, cap, H)
            s["slots"] = room(N, rows, k, dt=torch.int32)
            s["offsets"] = room(N, E // N + 1, dt=torch.int32)
        else:
            s["slots"] = _plan(ids, E, cap)[0]
            s["recv"] = normal(N, cap, H)
            s["weights"] = torch.rand(N, rows, k, generator=g, device="cuda")
            s["weights"] /= s["weights"].sum(-1, keepdim=True)
            if op == "combine":
                s["out"] = room(N, rows, H)
            else:
                s["dout"] = normal(N, rows, H)
                s["drecv"], s["dweights"] = room(N, cap, H), room(N, rows, k, dt=torch.float32)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _norm(s):
    h = s["send"].view(s["c"]["N"], *s["residual"].shape).float().sum(0) + s["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + EPS)
    y = h * rstd[..., None] * s["weight"].float()
    r = {"residual_out": h.to(s["residual"].dtype), "rstd": rstd}
    if not s["c"]["i8"]:
        return {**r, "out": y.to(s["residual"].dtype)}
    most = y.abs().amax(-1)
    scale = most / 127
    q = torch.clamp(torch.round(y * torch.where(most > 0, 127 / most, 0)[..., None]), -127, 127)
    return {**r, "out": (q * scale[..., None]).to(s["residual"].dtype), "scale": scale}


def _norm_backward(s):
    h, rstd, dy = s["h"].float(), s["rstd"][..., None], s["dout"].float()
    g = dy * s["weight"].float()
    dh = rstd * (g - h * (rstd * rstd * (g * h).mean(-1, keepdim=True))) + s["dresidual_out"].float()
    dw = (dy * h * rstd).sum(1)
    dh = dh.to(s["h"].dtype)
    every = dh.view(1, *s["dsend"].shape[1:]).expand(s["c"]["N"], -1, -1).contiguous()
    return {"dsend": every, "dresidual": dh, "dweight": dw}


def _pairs(x):
    """The sum over the last dimension, neighbours first."""
    return x if x.shape[-1] == 1 else _pairs(x[..., 0::2] + x[..., 1::2])


def _scores(l, score):
    """The experts' scores of logits in fp32; 0 where a logit is -inf or NaN."""
    there = l > -math.inf
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        most = torch.where(there, l, -math.inf).amax(-1, keepdim=True)
        e = torch.where(there, torch.where(l == most, 1.0, torch.exp(l - most)), 0.0)
        pad = 2 ** math.ceil(math.log2(l.shape[-1])) - l.shape[-1]
        s = e / _pairs(torch.nn.functional.pad(e, (0, pad)))
    return torch.where(there, s, 0.0)


def _route(s):
    c, l = s["c"], s["logits"].float()
    E, k, G = c["E"], c["k"], c["groups"]
    score = _scores(l, c["score"])
    by = score if s["bias"] is not None or (G > 1 and c["top"] == 2) else l
    if s["bias"] is not None:
        by = by + s["bias"]
    by = torch.where((l > -math.inf) & (by > -math.inf), by, -math.inf)
    if G > 1:
        best = torch.sort(by.view(*by.shape[:-1], G, E // G), dim=-1, descending=True)[0][..., :min(c["top"], E // G)]
        worth = best[..., 0]
        if best.shape[-1] == 2:
            worth = torch.where(best[..., 1] > -math.inf, best[..., 0] + best[..., 1], best[..., 0])
        kept = torch.sort(worth, dim=-1, descending=True, stable=True)[1][..., :c["keep"]]
        on = torch.zeros_like(worth, dtype=torch.bool).scatter(-1, kept, True)
        by = torch.where(on[..., None], by.view(*by.shape[:-1], G, E // G), -math.inf).view_as(by)
    top, ids = torch.sort(by, dim=-1, descending=True, stable=True)
    top, ids = top[..., :k], ids[..., :k]
    w = torch.where(top > -math.inf, torch.gather(score, -1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=TINY)
    return {"ids": torch.where(top > -math.inf, ids, -1).to(torch.int32), "weights": w * _scale(c)}


def _scale(c):
    return 2.5 if c["score"] == "sigmoid" else 1.0


def _route_backward(s):
    c, l = s["c"], s["logits"].float()
    score = _scores(l, c["score"])
    chosen = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    p = torch.where(chosen, torch.gather(score, -1, at), 0.0)
    d = torch.where(chosen, s["dweights"] * _scale(c), 0.0)
    if c["renorm"]:
        total = p.sum(-1, keepdim=True)
        d = torch.where(total >= TINY, (d - (d * p).sum(-1, keepdim=True) / total) / total, 0.0)
    ds = torch.zeros_like(score).scatter_add(-1, at, torch.where(chosen, d, 0.0))
    if c["score"] == "sigmoid":
        dl = ds * score * (1 - score)
    else:
        dl = score * (ds - (d * p).sum(-1, keepdim=True))
    return {"dlogits": dl.to(s["logits"].dtype)}


def _plan(ids, E, cap):
    """Where each (token, choice) goes: rank * cap + row on the rank that holds
    its expert, or -1; rows in the order (expert, source rank, token, choice).
    And the first row of each of a rank's experts, and the end of the last."""
    N = ids.shape[0]
    e = ids.reshape(-1).long()
    there = (e >= 0) & (e < E)
    key, order = torch.sort(torch.where(there, e, E), stable=True)
    first = torch.searchsorted(key, torch.arange(E + 1, device=ids.device))
    rank = key // (E // N)
    base = first[0::E // N]
    row = torch.arange(key.numel(), device=ids.device) - base[rank]
    slot = torch.where((key < E) & (row < cap), rank * cap + row, -1)
    slots = torch.empty_like(slot).scatter_(0, order, slot).to(torch.int32).view_as(ids)
    ends = torch.cat([first[:-1].view(N, -1), base[1:, None]], 1) - base[:-1, None]
    return slots, ends.clamp(max=cap).to(torch.int32)


def _sources(slots, total):
    """For each of `total` rows the (token, choice) that goes there, or -1."""
    a = torch.arange(slots.numel(), device=slots.device)
    to = torch.where(slots.reshape(-1) >= 0, slots.reshape(-1).long(), total)
    return torch.full((total + 1,), -1, device=slots.device).scatter_(0, to, a)[:total]


def _dispatch(s):
    c = s["c"]
    slots, offsets = _plan(s["ids"], c["E"], s["capacity"])
    src = _sources(slots, c["N"] * s["capacity"])
    token = src.clamp(min=0) // c["k"]
    rows = s["send"].view(-1, c["H"])[token].view_as(s["recv"])
    there = (src >= 0).view(c["N"], -1)
    r = {"slots": slots, "offsets": offsets, "recv": torch.where(there[..., None], rows, s["recv"])}
    if c["dt"] == "i8":
        r["recv_scale"] = torch.where(there, s["scale"].view(-1)[token].view_as(there), s["recv_scale"])
    return r


def _combine(s):
    c = s["c"]
    there = s["slots"] >= 0
    rows = s["recv"].view(-1, c["H"])[s["slots"].clamp(min=0).long()].float()
    w = torch.where(there, s["weights"], 0.0)
    return {"out": (torch.where(there[..., None], rows, 0.0) * w[..., None]).sum(-2).to(s["out"].dtype)}


def _combine_backward(s):
    c = s["c"]
    there = s["slots"] >= 0
    dout = s["dout"].float()
    rows = s["recv"].view(-1, c["H"])[s["slots"].clamp(min=0).long()].float()
    dw = torch.where(there, (rows * dout[..., None, :]).sum(-1), 0.0)
    src = _sources(s["slots"], c["N"] * s["recv"].shape[1])
    a = src.clamp(min=0)
    d = (dout.view(-1, c["H"])[a // c["k"]] * s["weights"].view(-1, 1)[a]).to(s["recv"].dtype).view_as(s["recv"])
    return {"drecv": torch.where((src >= 0).view(c["N"], -1, 1), d, s["drecv"]), "dweights": dw}


PLAIN = {"norm": _norm, "norm_bwd": _norm_backward, "route": _route, "route_bwd": _route_backward,
         "dispatch": _dispatch, "combine": _combine, "combine_bwd": _combine_backward}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import collective_communication_algorithms_virtual_gb300 as vc

    c, op = s["c"], s["c"]["op"]
    if op == "norm":
        vc.vc_reduce_scatter_norm(s["send"], s["weight"], s["out"], residual=s["residual"],
                                  residual_out=s["residual_out"], scale=s.get("scale"), rstd=s["rstd"], eps=EPS)
        r = {"residual_out": s["residual_out"], "rstd": s["rstd"], "out": s["out"]}
        if c["i8"]:  # as the values that the 8-bit numbers stand for
            r["out"] = torch.mul(s["out"], s["scale"][..., None], out=s["value"])
            r["scale"] = s["scale"]
        return r
    if op == "norm_bwd":
        vc.vc_reduce_scatter_norm_backward(s["dout"], s["h"], s["weight"], s["rstd"], dsend=s["dsend"],
                                           dresidual=s["dresidual"], dweight=s["dweight"],
                                           dresidual_out=s["dresidual_out"])
        return {"dsend": s["dsend"], "dresidual": s["dresidual"], "dweight": s["dweight"]}
    if op == "route":
        vc.vc_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], score=c["score"], ngroups=c["groups"],
                    topk_groups=c["keep"], group_top=c["top"], renormalize=c["renorm"], scale=_scale(c))
        return {"ids": s["ids"], "weights": s["weights"]}
    if op == "route_bwd":
        vc.vc_route_backward(s["dweights"], s["logits"], s["ids"], s["dlogits"], score=c["score"],
                             renormalize=c["renorm"], scale=_scale(c))
        return {"dlogits": s["dlogits"]}
    if op == "dispatch":
        vc.vc_dispatch_plan(s["ids"], s["slots"], s["offsets"], s["capacity"])
        vc.vc_dispatch(s["send"], s["slots"], s["recv"], scale=s.get("scale"), recv_scale=s.get("recv_scale"))
        r = {"slots": s["slots"], "offsets": s["offsets"], "recv": s["recv"]}
        return {**r, "recv_scale": s["recv_scale"]} if c["dt"] == "i8" else r
    if op == "combine":
        vc.vc_combine(s["recv"], s["slots"], s["out"], weights=s["weights"])
        return {"out": s["out"]}
    vc.vc_combine_backward(s["dout"], s["recv"], s["slots"], s["weights"], drecv=s["drecv"], dweights=s["dweights"])
    return {"drecv": s["drecv"], "dweights": s["dweights"]}


def run(state):
    return _own(state) if own else PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    N = c["N"]
    if op == "norm":
        T, H = N * c["rows"], c["H"]
        h = s["residual"].double().reshape(T, H)
        for q in range(N):
            h = h + s["send"][q].double()
        ms = torch.einsum("th,th->t", h, h) / H
        y = torch.einsum("th,t,h->th", h, (ms + EPS) ** -0.5, s["weight"].double())
        r = {"residual_out": h.view(N, -1, H), "rstd": ((ms + EPS) ** -0.5).view(N, -1), "out": y.view(N, -1, H)}
        if c["i8"]:
            # the nearest of 255 multiples of a 127th of the row's largest value
            top = torch.maximum(y.max(1).values, -y.min(1).values)
            step = (top / 127)[:, None]
            r["scale"] = step.view(N, -1)
            r["out"] = (torch.where(step > 0, torch.round(y / step), 0) * step).view(N, -1, H)
        return r
    if op == "norm_bwd":
        T, H = N * c["rows"], c["H"]
        h, dy, r = s["h"].double().view(T, H), s["dout"].double().view(T, H), s["rstd"].double().view(T)
        w = s["weight"].double()
        # y_i = w_i h_i r with dr/dh_j = -r^3 h_j / H
        along = torch.einsum("th,th,h->t", dy, h, w)
        dh = dy * w * r[:, None] - torch.einsum("t,th->th", r ** 3 * along / H, h) + s["dresidual_out"].double().view(T, H)
        dw = torch.einsum("nth,nth,nt->nh", dy.view(N, -1, H), h.view(N, -1, H), r.view(N, -1))
        return {"dsend": dh.repeat(N, 1, 1), "dresidual": dh.view(N, -1, H), "dweight": dw}
    if op == "route":
        l = s["logits"].double()
        sc = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
        by = (sc if s["bias"] is None else sc + s["bias"].double()).masked_fill(l == -math.inf, -math.inf)
        G, each = c["groups"], c["E"] // c["groups"]
        if G > 1:
            worth = torch.stack([by[..., g * each:(g + 1) * each].topk(min(c["top"], each)).values.sum(-1)
                                 for g in range(G)], -1)
            level, lower = worth[..., None, :] == worth[..., None], torch.ones(G, G, device="cuda").tril(-1).bool()
            place = ((worth[..., None, :] > worth[..., None]) | (level & lower)).sum(-1)
            by = by.masked_fill((place >= c["keep"]).repeat_interleave(each, -1), -math.inf)
        top, ids = by.sort(dim=-1, descending=True, stable=True)
        ids = ids.masked_fill(top == -math.inf, -1)[..., :c["k"]]
        w = torch.where(ids >= 0, sc.gather(-1, ids.long().clamp(min=0)), 0)
        if c["renorm"]:
            w = torch.where(ids >= 0, w / w.sum(-1, keepdim=True), 0)
        return {"ids": None, "weights": w * _scale(c)}
    if op == "route_bwd":
        l = s["logits"].double()
        live = (l > -math.inf).any(-1, keepdim=True)
        l = torch.where(live, l, 0).requires_grad_(True)
        sc = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
        w = torch.where(s["ids"] >= 0, sc.gather(-1, s["ids"].long().clamp(min=0)), 0)
        if c["renorm"]:
            w = torch.where(live, w / torch.where(live, w.sum(-1, keepdim=True), 1), 0)
        (w * _scale(c) * s["dweights"].double()).sum().backward()
        return {"dlogits": torch.where(live, l.grad, 0)}
    if op == "dispatch":
        # rows are moved, not computed: expert by expert, every token that chose it
        recv, e = s["recv"].double(), s["ids"].view(-1, c["k"])
        recv_scale = s["recv_scale"].double() if c["dt"] == "i8" else None
        each = c["E"] // N
        for d in range(N):
            t = torch.cat([torch.nonzero((e == d * each + i).any(1))[:, 0] for i in range(each)])[:s["capacity"]]
            recv[d, :t.numel()] = s["send"].reshape(-1, c["H"])[t].double()
            if recv_scale is not None:
                recv_scale[d, :t.numel()] = s["scale"].reshape(-1)[t].double()
        r = {"slots": None, "offsets": None, "recv": None if c["dt"] == "i8" else recv}
        return {**r, "recv_scale": recv_scale} if c["dt"] == "i8" else r
    slots, y = s["slots"].view(-1, c["k"]).long(), s["recv"].double().reshape(-1, c["H"])
    w = s["weights"].double().view(-1, c["k"])
    if op == "combine":
        out = torch.zeros(slots.shape[0], c["H"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            t = torch.nonzero(slots[:, j] >= 0)[:, 0]
            out[t] += w[t, j, None] * y[slots[t, j]]
        return {"out": out.view(N, -1, c["H"])}
    dout = s["dout"].double().view(-1, c["H"])
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(c["k"]):
        t = torch.nonzero(slots[:, j] >= 0)[:, 0]
        dy[slots[t, j]] = w[t, j, None] * dout[t]
        dw[t, j] = torch.einsum("th,th->t", dout[t], y[slots[t, j]])
    return {"drecv": dy.view(N, -1, c["H"]), "dweights": dw.view(N, -1, c["k"])}
