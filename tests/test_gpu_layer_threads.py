"""Layer operators from several host threads, each on its own stream, with
sizes that differ between the threads: the same bits as from one thread.

The first calls of the kernels whose shared memory goes by the call are made
in a process of their own, so that they race here."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import collective_communication_algorithms_virtual_gb300 as vc

from .conftest import ROOT

pytestmark = pytest.mark.gpu

THREADS = 4


def calls(tid):
    """One thread's calls: rows taken element by element, plans of many
    experts, and what else a layer does; returns their outputs."""
    g = torch.Generator().manual_seed(tid)
    dt = torch.bfloat16
    N, rows, H, E, k = 2, 6, 49152 - 4096 * tid - 1, 1024 - 128 * tid, 3
    found = []
    send = (torch.randn(N, N * rows, H, generator=g)).to(dt).cuda()
    res, w = torch.randn(N, rows, H, generator=g).to(dt).cuda(), torch.ones(H, dtype=dt, device="cuda")
    h, y, rs = torch.empty_like(res), torch.empty_like(res), torch.empty(N, rows, device="cuda")
    vc.vc_reduce_scatter_norm(send, w, y, residual=res, residual_out=h, rstd=rs)
    dres, dw = torch.empty_like(res), torch.empty(N, H, device="cuda")
    vc.vc_reduce_scatter_norm_backward(y, h, w, rs, dresidual=dres, dweight=dw)
    logits = torch.randn(N, 300, E, generator=g).cuda()
    ids, wt = torch.empty(N, 300, k, dtype=torch.int32, device="cuda"), torch.empty(N, 300, k, device="cuda")
    vc.vc_route(logits, ids, wt)
    slots, offsets = torch.empty_like(ids), torch.empty(N, E // N + 1, dtype=torch.int32, device="cuda")
    vc.vc_dispatch_plan(ids, slots, offsets, 600)
    x, recv = torch.randn(N, 300, 64 + tid, generator=g).cuda(), torch.zeros(N, 600, 64 + tid, device="cuda")
    vc.vc_dispatch(x, slots, recv)
    out = torch.empty_like(x)
    vc.vc_combine(recv, slots, out, weights=wt)
    found += [h, y, rs, dres, dw, ids, wt, slots, offsets, recv, out]
    return found


def race():
    torch.cuda.init()
    torch.zeros(1, device="cuda")
    vc.lib()
    found, errors, start = [None] * THREADS, [], threading.Barrier(THREADS)

    def work(tid):
        try:
            stream = torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(3):
                    found[tid] = calls(tid)
            stream.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append((tid, repr(e)))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for tid in range(THREADS):
        again = calls(tid)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(found[tid], again)), tid


def test_threads_of_different_sizes():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    code = "from tests.test_gpu_layer_threads import race; race(); print('ok')"
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT},
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.endswith("ok\n"), out.stderr[-2000:]
