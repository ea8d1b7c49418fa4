"""The layer operators together: the expert-parallel layer of examples/, the
launch trace's names, the device error word, and a large dispatch (the
bulk-copy path) against the same rows in torch.

The layer's distances from 64-bit torch: bf16 rounds each of about six stored
tensors on the way to 2^-9 rms, so an output and its gradients are within a
few times that, 2e-2; 8-bit tokens add a uniform error of a 127th of a row's
largest value (about 3.5 standard deviations), 0.8% rms, within 3e-2 with it.
In fp32 without 8 bits the torch products themselves round to 2^-11 (TF32 is
off by default), so 1e-4 holds with a wide margin."""
import importlib.util
import os

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("expert_parallel_layer",
                                                  os.path.join(ROOT, "examples", "expert_parallel_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("N,rows,hidden,experts,topk", [(4, 64, 512, 16, 4), (1, 5, 96, 4, 2), (3, 17, 200, 9, 3)])
def test_layer_matches_plain_torch(example, N, rows, hidden, experts, topk):
    for name, d in example.compare(N, rows, hidden, experts, topk).items():
        assert d <= (3e-2 if name == "serve" else 2e-2), (name, d)
    for name, d in example.compare(N, rows, hidden, experts, topk, torch.float32).items():
        assert d <= (3e-2 if name == "serve" else 1e-4), (name, d)


def test_launch_trace_names_the_kernels(example):
    layer = example.Layer(2, 8, 64, 4, 2)
    partial = torch.randn(2, 16, 64, device="cuda").bfloat16()
    residual, dout = torch.randn(2, 8, 64, device="cuda").bfloat16(), torch.randn(2, 8, 64, device="cuda").bfloat16()
    vc.vc_trace_enable(True)
    try:
        layer.train(partial, residual, dout)
        recs = vc.vc_trace_read()
    finally:
        vc.vc_trace_enable(False)
    own = [r for r in recs if r["coll"] == -1]
    assert [r["kernel"] for r in own] == ["norm", "route", "dispatch_plan", "dispatch", "combine", "combine_backward",
                                          "combine", "route_backward", "norm_backward", "norm_weight"]
    # partial sums, residual and weights in, residual and output out, 1/rms
    assert own[0]["bytes"] == 16 * 64 * 2 * (2 + 3) + 2 * 64 * 2 + 16 * 4
    assert all(r["ms"] > 0 for r in own)


@pytest.mark.parametrize("H,dt", [(4096, torch.bfloat16), (2056, torch.float32), (8208, torch.int8)])
def test_large_dispatch(example, H, dt):
    """Over 128 MiB of rows to five places each, some skipped."""
    N, rows, k, E = 2, 2100, 5, 10
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(-1, E, (N, rows, k), generator=g, device="cuda", dtype=torch.int32)
    cap = N * rows * k // N
    slots, offsets = torch.empty_like(ids), torch.empty(N, E // N + 1, dtype=torch.int32, device="cuda")
    vc.vc_dispatch_plan(ids, slots, offsets, cap)
    send = torch.randint(-100, 100, (N, rows, H), generator=g, device="cuda").to(dt)
    scale = torch.rand(N, rows, generator=g, device="cuda")
    recv, rscale = torch.zeros(N, cap, H, dtype=dt, device="cuda"), torch.zeros(N, cap, device="cuda")
    assert (slots >= 0).sum().item() * H * send.element_size() > 100 << 20 and N * rows * k * H * send.element_size() >= 128 << 20
    vc.vc_dispatch(send, slots, recv, scale=scale, recv_scale=rscale)
    on = torch.nonzero(slots.view(-1) >= 0)[:, 0]
    want, want_s = torch.zeros_like(recv).view(-1, H), torch.zeros_like(rscale).view(-1)
    want[slots.view(-1)[on].long()] = send.view(-1, H)[on // k]
    want_s[slots.view(-1)[on].long()] = scale.view(-1)[on // k]
    assert torch.equal(recv.view(-1, H), want) and torch.equal(rscale.view(-1), want_s)
    assert vc.vc_device_errors() == 0
