"""One expert-parallel transformer layer step over virtual ranks, with the
library's layer operators around the user's own matrix products.

N ranks hold `rows` tokens each and E / N experts each.  What arrives is every
rank's partial sums of the attention output (tensor parallelism); then

  1. vc_reduce_scatter_norm  partial sums + residual -> residual, norm
  2. vc_route                the router's logits -> experts and their weights
  3. vc_dispatch_plan, vc_dispatch   tokens to their experts' ranks
  4. the experts' products: torch.matmul in a loop that waits for the offsets,
     or, with library=True, vc_expert_product, which reads them on the device
  5. vc_combine              the experts' answers, weighted, back to the tokens

`serve` sends the tokens in 8 bits with a scale each; `serve8` multiplies in
8-bit floating point too, with a scale for each block of 128; `train` keeps the
data type and runs the whole chain backward; `clip` scales the experts'
gradients by their norm over all ranks.  The command compares them with plain
torch on the same numbers:

  python examples/expert_parallel_layer.py [--ranks 4] [--rows 64] [--hidden 512] [--experts 16] [--topk 4]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import collective_communication_algorithms_virtual_gb300 as vc  # noqa: E402

HOW = dict(score="softmax", renormalize=True)


class Layer:
    """Weights of one layer, and buffers sized for one batch shape."""

    def __init__(self, N, rows, hidden, experts, topk, dtype=torch.bfloat16, seed=0, library=False):
        self.library = library
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.N, self.rows, self.H, self.E, self.k, self.dtype = N, rows, hidden, experts, topk, dtype
        self.cap = N * rows * min(topk, experts // N)  # room for every choice

        def normal(*shape, by=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * by

        self.norm = (1 + normal(hidden, by=0.1)).to(dtype)
        self.router = normal(hidden, experts, by=hidden ** -0.5).to(dtype)
        self.up = normal(experts, hidden, hidden, by=hidden ** -0.5).to(dtype)
        self.i32 = dict(dtype=torch.int32, device="cuda")
        self.f32 = dict(dtype=torch.float32, device="cuda")
        self.data = dict(dtype=dtype, device="cuda")
        self.ids, self.slots = (torch.empty(N, rows, topk, **self.i32) for _ in range(2))
        self.weights = torch.empty(N, rows, topk, **self.f32)
        self.offsets = torch.empty(N, experts // N + 1, **self.i32)
        self.h = torch.empty(N, rows, hidden, **self.data)
        self.rstd, self.scale = (torch.empty(N, rows, **self.f32) for _ in range(2))
        self.out = torch.empty(N, rows, hidden, **self.data)

    def route(self, logits):
        vc.vc_route(logits, self.ids, self.weights, **HOW)
        vc.vc_dispatch_plan(self.ids, self.slots, self.offsets, self.cap)

    def experts(self, recv):
        """The experts' products on the rows each has received."""
        each, answer = self.E // self.N, torch.zeros(self.N, self.cap, self.H, **self.data)
        if self.library:
            vc.vc_expert_product(recv, self.up.view(self.N, each, self.H, self.H), self.offsets, answer)
            return answer
        for d, ends in enumerate(self.offsets.tolist()):
            for i in range(each):
                rows = slice(ends[i], ends[i + 1])
                answer[d, rows] = recv[d, rows] @ self.up[d * each + i]
        return answer

    def serve(self, partial, residual):
        """partial (N, N * rows, hidden), residual (N, rows, hidden) -> the
        layer's output; the new residual stream is in self.h."""
        N, rows, H = self.N, self.rows, self.H
        y8 = torch.empty(N, rows, H, dtype=torch.int8, device="cuda")
        vc.vc_reduce_scatter_norm(partial, self.norm, y8, residual=residual, residual_out=self.h, scale=self.scale)
        y = (y8.float() * self.scale[..., None]).to(self.dtype)
        self.route(y @ self.router)
        recv8 = torch.empty(N, self.cap, H, dtype=torch.int8, device="cuda")
        recv_scale = torch.zeros(N, self.cap, **self.f32)
        vc.vc_dispatch(y8, self.slots, recv8, scale=self.scale, recv_scale=recv_scale)
        recv = (recv8.float() * recv_scale[..., None]).to(self.dtype)
        vc.vc_combine(self.experts(recv), self.slots, self.out, weights=self.weights)
        return self.out

    def serve8(self, partial, residual):
        """As serve, the experts' products in 8-bit floating point."""
        N, rows, H, each = self.N, self.rows, self.H, self.E // self.N
        blocks, f8 = -(-H // vc.FP8_BLOCK), dict(dtype=torch.float8_e4m3fn, device="cuda")
        up = self.up.view(N, each, H, H).transpose(2, 3).contiguous()  # a program keeps these two
        up8, up_scale = torch.empty(N, each, H, H, **f8), torch.empty(N, each, blocks, blocks, **self.f32)
        vc.vc_quantize_fp8(up, up8, up_scale, block_rows=vc.FP8_BLOCK)
        y = torch.empty(N, rows, H, **self.data)
        vc.vc_reduce_scatter_norm(partial, self.norm, y, residual=residual, residual_out=self.h)
        self.route(y @ self.router)
        y8, scale = torch.empty(N, rows, H, **f8), torch.empty(N, rows, blocks, **self.f32)
        vc.vc_quantize_fp8(y, y8, scale)
        recv8, recv_scale = torch.empty(N, self.cap, H, **f8), torch.empty(N, self.cap, blocks, **self.f32)
        vc.vc_dispatch(y8, self.slots, recv8)
        vc.vc_dispatch(scale, self.slots, recv_scale)  # a row's scales go where the row goes
        answer = torch.empty(N, self.cap, H, **self.data)
        vc.vc_expert_product_fp8(recv8, recv_scale, up8, up_scale, self.offsets, answer)
        vc.vc_combine(answer, self.slots, self.out, weights=self.weights)
        return self.out

    def clip(self, grads, max_norm):
        """Scales the experts' gradients, each rank holding its own experts', in
        place where their norm over all ranks is above max_norm; the norm."""
        each, norm = self.E // self.N, torch.empty(self.N, **self.f32)
        vc.vc_clip_grad_norm([[grads["up"][r * each:(r + 1) * each]] for r in range(self.N)], norm, max_norm=max_norm)
        return norm

    def train(self, partial, residual, dout):
        """Forward in the data type, then the gradients of
        sum(out * dout): a dict of them."""
        N, rows, H, each = self.N, self.rows, self.H, self.E // self.N
        y = torch.empty(N, rows, H, **self.data)
        vc.vc_reduce_scatter_norm(partial, self.norm, y, residual=residual, residual_out=self.h, rstd=self.rstd)
        logits = y @ self.router
        self.route(logits)
        recv = torch.zeros(N, self.cap, H, **self.data)
        vc.vc_dispatch(y, self.slots, recv)
        answer = self.experts(recv)
        vc.vc_combine(answer, self.slots, self.out, weights=self.weights)

        danswer, dweights = torch.zeros_like(answer), torch.empty_like(self.weights)
        vc.vc_combine_backward(dout, answer, self.slots, self.weights, drecv=danswer, dweights=dweights)
        drecv, dup = torch.zeros_like(recv), torch.zeros_like(self.up)
        if self.library:
            experts = (N, each, H, H)
            vc.vc_expert_product_backward(danswer, recv, self.up.view(experts), self.offsets, drows=drecv, dweight=dup.view(experts))
        for d, ends in enumerate([] if self.library else self.offsets.tolist()):
            for i in range(each):
                at, e = slice(ends[i], ends[i + 1]), d * each + i
                drecv[d, at] = danswer[d, at] @ self.up[e].T
                dup[e] = recv[d, at].T @ danswer[d, at]
        dy = torch.empty_like(y)
        vc.vc_combine(drecv, self.slots, dy)  # dispatch's gradient
        dlogits = torch.empty_like(logits)
        vc.vc_route_backward(dweights, logits, self.ids, dlogits, **HOW)
        dy += dlogits @ self.router.T
        drouter = y.reshape(-1, H).T @ dlogits.reshape(-1, self.E)
        dpartial, dresidual = torch.empty_like(partial), torch.empty_like(residual)
        dnorm = torch.empty(N, H, **self.f32)
        vc.vc_reduce_scatter_norm_backward(dy, self.h, self.norm, self.rstd, dsend=dpartial, dresidual=dresidual,
                                           dweight=dnorm)
        vc.vc_allreduce(list(dnorm), list(dnorm))  # each rank's part to the whole, on every rank
        return {"partial": dpartial, "residual": dresidual, "norm": dnorm[0], "router": drouter, "up": dup}


def plain(layer, partial, residual, ids, dtype=torch.float64):
    """The layer in plain torch for given experts, in 64 bits."""
    N, rows, H = residual.shape
    x = partial.to(dtype).view(N, N, rows, H).sum(0) + residual.to(dtype)
    y = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * layer["norm"]
    s = torch.softmax(y @ layer["router"], -1)
    w = s.gather(-1, ids.long())
    w = w / w.sum(-1, keepdim=True)
    every = torch.einsum("nth,ehk->ntek", y, layer["up"])
    return (every.gather(2, ids.long()[..., None].expand(-1, -1, -1, H)) * w[..., None]).sum(2)


def distance(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def compare(N=4, rows=64, hidden=512, experts=16, topk=4, dtype=torch.bfloat16, library=False):
    """Relative distances of the layer's output and gradients from plain torch."""
    layer = Layer(N, rows, hidden, experts, topk, dtype, library=library)
    g = torch.Generator(device="cuda").manual_seed(1)
    partial = (torch.randn(N, N * rows, hidden, generator=g, device="cuda") * N ** -0.5).to(dtype)
    residual = torch.randn(N, rows, hidden, generator=g, device="cuda").to(dtype)
    dout = torch.randn(N, rows, hidden, generator=g, device="cuda").to(dtype)
    found = {}
    out = layer.serve(partial, residual).clone()
    weights = {"norm": layer.norm, "router": layer.router, "up": layer.up}
    leaves = {k: v.double().requires_grad_(True) for k, v in {**weights, "partial": partial, "residual": residual}.items()}
    found["serve"] = distance(out, plain(leaves, leaves["partial"], leaves["residual"], layer.ids).detach())
    grads = layer.train(partial, residual, dout)
    want = plain(leaves, leaves["partial"], leaves["residual"], layer.ids)
    found["train"] = distance(layer.out, want.detach())
    (want * dout.double()).sum().backward()
    for k, v in grads.items():
        found["d" + k] = distance(v, leaves[k].grad)
    if library:
        out = layer.serve8(partial, residual)
        found["serve8"] = distance(out, plain(leaves, leaves["partial"], leaves["residual"], layer.ids).detach())
        whole = leaves["up"].grad
        norm = layer.clip(grads, float(whole.norm()) / 2)
        found["norm"] = float((norm.double() - whole.norm()).abs().max() / whole.norm())
        found["clipped"] = distance(grads["up"], whole / 2)
    return found


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("ranks", 4), ("rows", 64), ("hidden", 512), ("experts", 16), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    for library in (False, True):
        print("products of the library" if library else "products in torch")
        for k, v in compare(a.ranks, a.rows, a.hidden, a.experts, a.topk, library=library).items():
            print(f"  {k:10s} relative distance from plain torch {v:.2e}")
