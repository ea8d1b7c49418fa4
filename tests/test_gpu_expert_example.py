"""The experts' operators in the expert-parallel layer of examples/: routing,
dispatch, products, combine and the gradients together, in 16 and 8 bits, and
the clipping of the experts' gradients.

The distances are those of the products in torch (tests/test_gpu_layer_example.py):
2e-2 for bf16, 1e-4 for fp32.  In 8 bits rows and weights are off by at most
2^-4 of each element, spread over a step: 2.6% rms each, 3.7% of a product of
independent sums, so within 6e-2 with the bf16 roundings.  The norm of gradients
within 2e-2 of theirs is within 2e-2 too."""
import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .test_gpu_layer_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,rows,hidden,experts,topk", [(4, 64, 512, 16, 4), (1, 5, 96, 4, 2), (3, 17, 200, 9, 3)])
def test_layer_with_the_librarys_products(example, N, rows, hidden, experts, topk):  # noqa: F811
    for name, d in example.compare(N, rows, hidden, experts, topk, library=True).items():
        assert d <= {"serve": 3e-2, "serve8": 6e-2}.get(name, 2e-2), (name, d)
    for name, d in example.compare(N, rows, hidden, experts, topk, torch.float32, library=True).items():
        assert d <= {"serve": 3e-2, "serve8": 6e-2}.get(name, 1e-4), (name, d)
    assert vc.vc_device_errors() == 0


def test_launch_trace_names_the_products(example):  # noqa: F811
    layer = example.Layer(2, 8, 64, 4, 2, library=True)
    partial = torch.randn(2, 16, 64, device="cuda").bfloat16()
    residual, dout = torch.randn(2, 8, 64, device="cuda").bfloat16(), torch.randn(2, 8, 64, device="cuda").bfloat16()
    vc.vc_trace_enable(True)
    try:
        grads = layer.train(partial, residual, dout)
        layer.clip(grads, 1e-3)
        layer.serve8(partial, residual)
        recs = vc.vc_trace_read()
    finally:
        vc.vc_trace_enable(False)
    own = [r["kernel"] for r in recs if r["coll"] == -1]
    assert own == ["norm", "route", "dispatch_plan", "dispatch", "expert_product", "combine", "combine_backward",
                   "expert_product", "expert_weight", "combine", "route_backward", "norm_backward", "norm_weight", "grad_norm",
                   "clip", "quantize", "norm", "route", "dispatch_plan", "quantize", "dispatch", "dispatch",
                   "expert_product_fp8", "combine"]


def test_products_captured_with_their_neighbours(example):  # noqa: F811
    """One graph from the routing to the combined answers; other tokens in the
    same buffers change the experts' rows, and the replay follows."""
    layer = example.Layer(2, 40, 256, 8, 2, library=True)
    y = torch.randn(2, 40, 256, device="cuda").bfloat16()
    recv, answer = (torch.zeros(2, layer.cap, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    logits = torch.empty(2, 40, 8, dtype=torch.bfloat16, device="cuda")

    def go():
        layer.route(logits)
        vc.vc_dispatch(y, layer.slots, recv)
        vc.vc_expert_product(recv, layer.up.view(2, 4, 256, 256), layer.offsets, answer)
        vc.vc_combine(answer, layer.slots, layer.out, weights=layer.weights)
    logits.copy_(y @ layer.router)
    go()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go()
    for seed in range(3):
        y.copy_(torch.randn(2, 40, 256, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        logits.copy_(y @ layer.router)
        graph.replay()
        torch.cuda.synchronize()
        got = layer.out.clone()
        go()
        torch.cuda.synchronize()
        assert torch.equal(got, layer.out)
