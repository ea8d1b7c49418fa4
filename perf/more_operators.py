"""Cases of the operators around an expert's weights: the products of the rows
that dispatch brought with the weights of their experts (and their gradients),
the same in 8-bit floating point with a scale for each block of 128, the
rounding to that form, and the clipping of the gradients by their global norm.

Each case names an operator ("op") and its sizes.  With ``own`` false, run()
computes it in elementary torch operations in fp32; with ``own`` true it calls
the library.  Every rank's buffers are slices of one tensor whose first
dimension is the virtual ranks.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
MOST8 = 448.0  # the largest e4m3 number
BLOCK = 128
MAX_NORM = 1.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The expert-parallel example's layer (4 ranks of 64 tokens): latency.
        {"name": "product-small", "op": "product", "N": 4, "rows": 64, "k": 4, "E": 16, "in": 512, "out": 512,
         "dt": "bf16", "transposed": False},
        # Four new tokens a rank during generation: the weights of 64 experts
        # are read for a few rows each.
        {"name": "product-decode", "op": "product", "N": 8, "rows": 4, "k": 4, "E": 64, "in": 4096, "out": 2048,
         "dt": "bf16", "transposed": True},
        # A prompt's 4096 tokens, eight experts each.
        {"name": "product-prefill", "op": "product", "N": 8, "rows": 512, "k": 8, "E": 64, "in": 4096, "out": 2048,
         "dt": "bf16", "transposed": True},
        # Odd widths and rank count (rows start off 16-byte boundaries).
        {"name": "product-odd-f16", "op": "product", "N": 5, "rows": 77, "k": 3, "E": 20, "in": 1003, "out": 515,
         "dt": "f16", "transposed": False},
        # The gradients of a training micro-batch's rows and of the weights.
        {"name": "product-backward", "op": "product_bwd", "N": 4, "rows": 1024, "k": 4, "E": 32, "in": 2048,
         "out": 4096, "dt": "bf16", "transposed": False},
        # Generation with 8-bit weights: half the bytes.
        {"name": "fp8-decode", "op": "fp8", "N": 8, "rows": 4, "k": 4, "E": 64, "in": 4096, "out": 2048, "dt": "bf16"},
        # A prompt in 8 bits: twice the rate.
        {"name": "fp8-prefill", "op": "fp8", "N": 8, "rows": 512, "k": 8, "E": 64, "in": 4096, "out": 2048,
         "dt": "bf16"},
        # New tokens to 8 bits before they are dispatched: latency.
        {"name": "quantize-decode", "op": "quantize", "N": 8, "rows": 4, "H": 4096, "dt": "bf16", "ragged": False,
         "each": 1, "block": 1},
        # The rows that each rank's experts have received, between two
        # products: bandwidth.
        {"name": "quantize-prefill", "op": "quantize", "N": 8, "rows": 5120, "H": 4096, "dt": "bf16", "ragged": True,
         "each": 8, "block": 1},
        # Weights to 8 bits, a scale for each 128 x 128, after an update.
        {"name": "quantize-weights", "op": "quantize", "N": 8, "rows": 2048, "H": 4096, "dt": "bf16", "ragged": False,
         "each": 8, "block": BLOCK},
        # The gradients of two small layers, a copy on each rank: latency.
        {"name": "clip-small", "op": "clip", "N": 4, "layers": 2, "H": 512, "F": 1024, "dt": "bf16", "across": False,
         "clips": True},
        # 24 layers' gradients, each rank holding its eighth of every tensor
        # after a ReduceScatter: bandwidth.
        {"name": "clip-large", "op": "clip", "N": 8, "layers": 24, "H": 2048, "F": 8192, "dt": "bf16", "across": True,
         "clips": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log(rng, lo, hi)
    return rng.choice([n, max(lo, n // 8 * 8), max(lo, n // 64 * 64), max(lo, n // 128 * 128)])


def _fit(case, by):
    """`case` made smaller where it would cost more than the largest listed
    one of its operator."""
    sizes = [work(c) for c in listed() if c["op"] == case["op"]]
    most = {k: max(s[k] for s in sizes) for k in ("bytes", "flops")}
    while any(work(case)[k] > most[k] for k in most):
        name = max(by, key=lambda n: case[n])
        if name == "E":
            case["E"] = max(case["N"], case["E"] // 2 // case["N"] * case["N"])
            case["k"] = min(case["k"], case["E"])
            by = [n for n in by if n != "E"] if case["E"] == case["N"] else by
        else:
            case[name] = max(1, case[name] * 3 // 4)
    return case


def draw(rng):
    op = rng.choice(["product", "product", "product", "product_bwd", "product_bwd", "fp8", "fp8", "quantize",
                     "quantize", "clip", "clip"])
    N = rng.choice([1, 2, 3, 4, 6, 8])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op in ("product", "product_bwd", "fp8"):
        E = N * _log(rng, 1, 64 // N)
        c = {"op": op, "N": N, "rows": _log(rng, 1, 2048), "k": min(E, rng.choice([1, 2, 4, 6, 8])), "E": E,
             "in": _width(rng, 64, 8192), "out": _width(rng, 64, 8192), "dt": dt}
        if op != "fp8":
            c["transposed"] = rng.random() < 0.5
        return _fit(c, ["rows", "in", "out", "E"])
    if op == "quantize":
        block = rng.choice([1, 1, BLOCK])
        c = {"op": op, "N": N, "rows": _log(rng, 1, 8192), "H": _width(rng, 64, 8192), "dt": dt,
             "ragged": block == 1 and rng.random() < 0.5, "each": _log(rng, 1, 8), "block": block}
        if block == 1 and not c["ragged"]:
            c["each"] = 1
        return _fit(c, ["rows", "H"])
    c = {"op": op, "N": N, "layers": _log(rng, 1, 32), "H": _width(rng, 64, 2048), "F": _width(rng, 64, 8192),
         "dt": rng.choice(["bf16", "f16", "f32"]), "across": rng.random() < 0.5, "clips": rng.random() < 0.7}
    return _fit(c, ["layers", "H", "F"])


def _size(dt):
    return {"f32": 4, "bf16": 2, "f16": 2}[dt]


def work(case):
    c, op = case, case["op"]
    N, es = c["N"], _size(c["dt"])
    if op in ("product", "product_bwd", "fp8"):
        T, I, O = N * c["rows"] * c["k"], c["in"], c["out"]
        # the experts that the rows reach, were every expert as likely
        met = c["E"] * (1 - (1 - 1 / c["E"]) ** T)
        ends = (c["E"] + N) * 4
        if op == "product":
            return {"bytes": T * (I + O) * es + met * I * O * es + ends, "flops": 2 * T * I * O}
        if op == "product_bwd":  # rows, their gradients' input and output, weights in, every weight's gradient out
            return {"bytes": T * (2 * I + O) * es + (met + c["E"]) * I * O * es + ends, "flops": 4 * T * I * O}
        blocks = -(-I // BLOCK)
        return {"bytes": T * (I + 4 * blocks + O * es) + met * (I * O + 4 * blocks * -(-O // BLOCK)) + ends,
                "flops": 2 * T * I * O}
    if op == "quantize":
        n = N * c["rows"] * (1 if c["ragged"] else c["each"])
        if c["ragged"]:
            n = n * 4 / 5  # what the experts have received of the room
        return {"bytes": n * c["H"] * (es + 1) + 4 * n / c["block"] * -(-c["H"] // BLOCK), "flops": 4 * n * c["H"]}
    n = c["layers"] * (4 * c["H"] ** 2 + 2 * c["H"] * c["F"]) * (1 if c["across"] else N)
    small = c["layers"] * 2 * c["H"] * (1 if c["across"] else N)
    return {"bytes": 2 * (n * es + small * 4) + 4 * N, "flops": 3 * (n + small)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _offsets(c, g, cap):
    """Where each rank's experts' rows begin, some experts more popular than
    others; what goes over the capacity is dropped."""
    E, N = c["E"], c["N"]
    liking = torch.softmax(torch.randn(E, generator=g, device="cuda") * 0.3, 0)
    picks = torch.multinomial(liking, N * c["rows"] * c["k"], replacement=True, generator=g)
    counts = torch.zeros(E, device="cuda").index_add_(0, picks, torch.ones(picks.numel(), device="cuda"))
    ends = torch.nn.functional.pad(counts.view(N, -1).cumsum(1), (1, 0)).clamp(max=cap)
    return ends.to(torch.int32).contiguous()


def _capacity(c):
    """Rows a rank has room for: every row where that is little, else a
    quarter above the mean."""
    T = c["N"] * c["rows"] * c["k"]
    return min(T, max(256, -(-5 * T // (4 * c["N"]))))


def _shards(c):
    """Elements of each rank's part of every tensor of the data type, and of
    the norms' weights in fp32; (ranks, tensors) each."""
    N, H, F = c["N"], c["H"], c["F"]
    big, small = [H * H] * 4 + [H * F] * 2, [H] * 2

    def parts(sizes):
        return [[n if not c["across"] else n // N + (r < n % N) for n in sizes] * c["layers"] for r in range(N)]
    return parts(big), parts(small)


def _views(flat, parts):
    """The tensors of each rank, one behind another in its buffer."""
    return [list(torch.split(flat[r, :sum(p)], p)) for r, p in enumerate(parts)]


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dt=None, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(dt or DT[c["dt"]])

    def room(*shape, dt=None):
        return torch.zeros(*shape, dtype=dt or DT[c["dt"]], device="cuda")

    N = c["N"]
    s = {"c": c}
    if op in ("product", "product_bwd", "fp8"):
        I, O, each, cap = c["in"], c["out"], c["E"] // N, _capacity(c)
        s["offsets"] = _offsets(c, g, cap)
        s["longest"] = max(1, int((s["offsets"][:, 1:] - s["offsets"][:, :-1]).max()))  # rows of one expert
        s["rows"] = normal(N, cap, I)
        shape = (O, I) if c.get("transposed", True) else (I, O)
        s["weight"] = torch.stack([normal(each, *shape, by=I ** -0.5) for _ in range(N)])
        if op == "product":
            s["out"] = room(N, cap, O)
        elif op == "product_bwd":
            s["dout"] = normal(N, cap, O)
            s["drows"], s["dweight"] = room(N, cap, I), torch.empty_like(s["weight"])
        else:
            s["rows"], s["row_scale"] = _quantized(s["rows"].float(), 1)
            q = [_quantized(w.float(), BLOCK) for w in s["weight"]]
            s["weight"], s["weight_scale"] = torch.stack([a for a, _ in q]), torch.stack([b for _, b in q])
            s["out"] = room(N, cap, O)
    elif op == "quantize":
        rows, H, mats = c["rows"], c["H"], 1 if c["ragged"] else c["each"]
        # rows of different size, as a layer's activations have them
        s["x"] = torch.stack([normal(mats, rows, H) for _ in range(N)])
        s["x"] *= torch.exp(torch.randn(N, mats, rows, 1, generator=g, device="cuda")).to(s["x"].dtype)
        s["out"] = room(N, mats, rows, H, dt=F8)
        s["scale"] = room(N, mats, -(-rows // c["block"]), -(-H // BLOCK), dt=torch.float32)
        s["offsets"] = None
        if c["ragged"]:
            part = torch.rand(N, c["each"], generator=g, device="cuda") + 0.5
            ends = (torch.nn.functional.pad(part.cumsum(1) / part.sum(1, keepdim=True), (1, 0)) * (rows * 4 // 5)).round()
            s["offsets"] = ends.to(torch.int32).contiguous()
    else:
        big, small = _shards(c)
        s["big"] = normal(N, max(map(sum, big)), by=1e-3)
        s["small"] = normal(N, max(map(sum, small)), dt=torch.float32, by=1e-2)
        s["big_out"], s["small_out"] = torch.empty_like(s["big"]), torch.empty_like(s["small"])
        s["tail"] = [(sum(b), sum(m)) for b, m in zip(big, small)]
        for b, m, (nb, nm) in zip(s["big"], s["small"], s["tail"]):  # shorter ranks' buffers end in zeros
            b[nb:], m[nm:] = 0, 0
        s["big_out"].zero_(), s["small_out"].zero_()
        s["grads"] = [a + b for a, b in zip(_views(s["big"], big), _views(s["small"], small))]
        s["outs"] = [a + b for a, b in zip(_views(s["big_out"], big), _views(s["small_out"], small))]
        s["norm"] = room(N, dt=torch.float32)
        s["max_norm"] = MAX_NORM * (1e-2 if c["clips"] else 1e6)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _grouped(s, rows):
    """The rows as (experts, longest, width), zeros behind each expert's last;
    and each row's place there, or one place more for rows of no expert."""
    N, cap, width = rows.shape
    ends = s["offsets"].long()
    each = ends.shape[1] - 1
    p = torch.arange(cap, device=rows.device).expand(N, cap).contiguous()
    e = torch.searchsorted(ends, p, right=True) - 1
    there = e < each
    e = e.clamp(max=each - 1)
    expert = torch.arange(N, device=rows.device)[:, None] * each + e
    at = torch.where(there, expert * s["longest"] + p - torch.gather(ends, 1, e), N * each * s["longest"])
    room = torch.zeros(N * each * s["longest"] + 1, width, device=rows.device)
    room[at.view(-1)] = rows.float().view(-1, width)
    return room[:-1].view(N * each, s["longest"], width), at, there


def _back(y, at, there, out):
    """(experts, longest, width) back to the rows; rows of no expert as `out` has them."""
    rows = y.reshape(-1, y.shape[-1])[at.clamp(max=y.shape[0] * y.shape[1] - 1)]
    return torch.where(there[..., None], rows.to(out.dtype), out)


def _weights(s):
    """(experts, in, out) in fp32."""
    w = s["weight"].flatten(0, 1).float()
    return w.transpose(1, 2) if s["c"].get("transposed", True) else w


def _product(s):
    x, at, there = _grouped(s, s["rows"])
    return {"out": _back(torch.bmm(x, _weights(s)), at, there, s["out"])}


def _product_backward(s):
    x, at, there = _grouped(s, s["rows"])
    dy = _grouped(s, s["dout"])[0]
    drows = _back(torch.bmm(dy, _weights(s).transpose(1, 2)), at, there, s["drows"])
    dw = torch.bmm(dy.transpose(1, 2), x) if s["c"]["transposed"] else torch.bmm(x.transpose(1, 2), dy)
    return {"drows": drows, "dweight": dw.to(s["weight"].dtype).view_as(s["dweight"])}


def _every(scale, dim, n):
    """A block's scale for each of the n elements along `dim`."""
    return scale.repeat_interleave(BLOCK, dim)[(slice(None),) * dim + (slice(n),)]


def _product_fp8(s):
    rows = s["rows"].float() * _every(s["row_scale"], 2, s["c"]["in"])
    x, at, there = _grouped(s, rows)
    scale = _every(_every(s["weight_scale"], 2, s["c"]["out"]), 3, s["c"]["in"])
    w = (s["weight"].float() * scale).flatten(0, 1).transpose(1, 2)
    return {"out": _back(torch.bmm(x, w), at, there, s["out"])}


def _quantized(x, block):
    """x (..., rows, width) in fp32 to e4m3 with a scale for each `block` rows
    and 128 of the width; scales are at least the smallest normal number but
    for blocks of zeros."""
    rows, width = x.shape[-2:]
    up, across = -rows % block, -width % BLOCK
    y = torch.nn.functional.pad(x, (0, across, 0, up))
    y = y.view(*x.shape[:-2], (rows + up) // block, block, (width + across) // BLOCK, BLOCK)
    most = y.abs().amax((-3, -1), keepdim=True)
    scale = torch.where(most > 0, (most / MOST8).clamp(min=2.0 ** -126), 0.0)
    q = (y * (MOST8 / most).clamp(max=2.0 ** 126)).clamp(-MOST8, MOST8)
    q = q.view(*x.shape[:-2], rows + up, width + across)[..., :rows, :width]
    return q.to(F8), scale[..., :, 0, :, 0].contiguous()


def _quantize(s):
    q, scale = _quantized(s["x"].float(), s["c"]["block"])
    if s["offsets"] is not None:  # rows behind the last expert's stay
        there = torch.arange(s["c"]["rows"], device=q.device) < s["offsets"][:, -1:]
        q = torch.where(there[:, None, :, None], q.float(), s["out"].float()).to(F8)
        scale = torch.where(there[:, None, :, None], scale, s["scale"])
    return {"out": q, "scale": scale}


def _clip(s):
    total = (s["big"].float().square().sum(1, dtype=torch.float64)
             + s["small"].square().sum(1, dtype=torch.float64))
    if s["c"]["across"]:
        total = total.sum().expand(len(total))
    norm = total.sqrt().float()
    by = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)[:, None]
    return {"big": (s["big"].float() * by).to(s["big"].dtype), "small": s["small"] * by, "norm": norm}


PLAIN = {"product": _product, "product_bwd": _product_backward, "fp8": _product_fp8, "quantize": _quantize,
         "clip": _clip}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import collective_communication_algorithms_virtual_gb300 as vc

    c, op = s["c"], s["c"]["op"]
    if op == "product":
        vc.vc_expert_product(s["rows"], s["weight"], s["offsets"], s["out"], transposed=c["transposed"])
        return {"out": s["out"]}
    if op == "product_bwd":
        vc.vc_expert_product_backward(s["dout"], s["rows"], s["weight"], s["offsets"], drows=s["drows"],
                                      dweight=s["dweight"], transposed=c["transposed"])
        return {"drows": s["drows"], "dweight": s["dweight"]}
    if op == "fp8":
        vc.vc_expert_product_fp8(s["rows"], s["row_scale"], s["weight"], s["weight_scale"], s["offsets"], s["out"])
        return {"out": s["out"]}
    if op == "quantize":
        vc.vc_quantize_fp8(s["x"], s["out"], s["scale"], offsets=s["offsets"], block_rows=c["block"])
        return {"out": s["out"], "scale": s["scale"]}
    vc.vc_clip_grad_norm(s["grads"], s["norm"], max_norm=s["max_norm"], out=s["outs"], across=c["across"])
    return {"big": s["big_out"], "small": s["small_out"], "norm": s["norm"]}


def run(state):
    return _own(state) if own else PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _blocks(n):
    return [(i // BLOCK, slice(i, min(n, i + BLOCK))) for i in range(0, n, BLOCK)]


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    N = c["N"]
    if op in ("product", "product_bwd", "fp8"):
        ends, r = s["offsets"].tolist(), {}
        if op == "product_bwd":
            r = {"drows": s["drows"].double(), "dweight": s["dweight"].double().zero_()}
        else:
            r = {"out": s["out"].double()}
        for d in range(N):
            for e, (lo, hi) in enumerate(zip(ends[d], ends[d][1:])):
                if lo == hi:
                    continue
                x, w = s["rows"][d, lo:hi].double(), s["weight"][d, e].double()
                if op == "product":
                    r["out"][d, lo:hi] = x @ (w.T if c["transposed"] else w)
                elif op == "product_bwd":
                    dy = s["dout"][d, lo:hi].double()
                    r["drows"][d, lo:hi] = dy @ (w if c["transposed"] else w.T)
                    r["dweight"][d, e] = dy.T @ x if c["transposed"] else x.T @ dy
                else:
                    for i, at in _blocks(c["in"]):
                        x[:, at] *= s["row_scale"][d, lo:hi, i, None].double()
                        for j, to in _blocks(c["out"]):
                            w[to, at] *= s["weight_scale"][d, e, j, i].double()
                    r["out"][d, lo:hi] = x @ w.T
        return r
    if op == "quantize":
        out, scale = s["out"].to(torch.float64), s["scale"].double()
        B = c["block"]
        last = [c["rows"]] * N if s["offsets"] is None else s["offsets"][:, -1].tolist()
        for d in range(N):
            x = s["x"][d].double()
            for i, at in _blocks(c["H"]):
                for lo in range(0, last[d], max(1, last[d]) if B == 1 else B):
                    to = slice(lo, last[d] if B == 1 else min(lo + B, last[d]))
                    part = x[:, to, at]
                    top = part.abs().amax(-1) if B == 1 else part.abs().flatten(1).amax(1, keepdim=True)
                    scale[d, :, to if B == 1 else slice(lo // B, lo // B + 1), i] = top / 448
                    out[d, :, to, at] = torch.where(top > 0, 448 / top, 0)[..., None] * part
        return {"out": out, "scale": scale}
    squares = torch.zeros(N, dtype=torch.float64, device="cuda")
    for r in range(N):
        for t in s["grads"][r]:
            squares[r] += torch.linalg.vector_norm(t.double()) ** 2
    if c["across"]:
        squares[:] = squares.sum()
    norm = squares ** 0.5
    factor = torch.minimum(s["max_norm"] / norm, torch.ones_like(norm))
    return {"big": s["big"].double() * factor[:, None], "small": s["small"].double() * factor[:, None], "norm": norm}
