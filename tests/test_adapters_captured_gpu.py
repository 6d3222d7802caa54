"""The operators of include/q4gsw_adapters.h inside CUDA graphs: the first calls of a process captured, ids that
change between replays, and two graphs that replay in turn."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALL_CAPTURED = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import bit_group_quantized_q4gsw_b200 as q
torch.manual_seed(0)
N, K, gs, L, r = 264, 512, 32, 3, 16
codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda")
blob = q.q4gsw_prepack(codes, (torch.rand(K // gs, N, device="cuda") * 0.01).half(), gs)
a, b = torch.randn(L, r, K, device="cuda").half() * 0.05, torch.randn(L, N, r, device="cuda").half() * 0.05
s = torch.rand(L, device="cuda") + 0.5
w, gate = torch.rand(K, device="cuda").half(), torch.rand(K, device="cuda").half()
few, many = [torch.randn(n, device="cuda") for n in (100, 5000)], [torch.randn(n, device="cuda") for n in (90000, 7)]
sets = [q.q4gsw_grad_set(g, [torch.empty_like(t) for t in g]) for g in (few, many)]
for M in (1, 12, 100, 1200):
    x, blk = torch.randn(M, K, device="cuda").half(), torch.randn(M, K, device="cuda").half()
    d = torch.randn(M, N, device="cuda").half() * 0.01
    ids = (torch.arange(M, device="cuda") % (L + 1) - 1).int()
    def step():
        plan = q.q4gsw_adapters_plan(ids, L)
        n, h = q.q4gsw_norms_fwd(x, block=blk, w_post=w, gate=gate, w_pre=w)
        y, u = q.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, n, scale=s, save_u=True)
        g = q.q4gsw_adapters_bwd(blob, N, K, gs, plan, a, b, n, u, d, scale=s)
        g += tuple(q.q4gsw_norms_bwd(h, d_x=g[0], block=blk, w_post=w, gate=gate, w_pre=w, want_weights=True))
        return (n, h, y, u) + g + tuple(q.q4gsw_grad_clip(t, 1.0) for t in sets) + tuple(q.q4gsw_grad_norm(t) for t in sets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):          # the first call of every kernel of this batch size
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, e) for p, e in zip(captured, step())), M
q.q4gsw_device_error_check()
print("first calls captured ok")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "first calls captured ok" in r.stdout


@pytest.mark.parametrize("M", [5, 16, 300, 1300])
def test_ids_change_between_replays_and_two_graphs_take_turns(M):
    # a plan inside the graph follows the ids of each replay, whatever their tiles; the graphs share operands and have
    # their own workspaces
    import bit_group_quantized_q4gsw_b200 as q
    N, K, gs, L, r = 136, 576, 64, 5, 24
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    blob = q.q4gsw_prepack(codes, torch.rand(K // gs, N, device="cuda", generator=g).half(), gs)
    a, b = (torch.randn(*s, device="cuda", generator=g).half() for s in ((L, r, K), (L, N, r)))
    x, d = torch.randn(M, K, device="cuda", generator=g).half(), torch.randn(M, N, device="cuda", generator=g).half()
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")

    def step():
        plan = q.q4gsw_adapters_plan(ids, L)
        y, u = q.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, x, save_u=True)
        return (y, u, *q.q4gsw_adapters_bwd(blob, N, K, gs, plan, a, b, x, u, d))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for i in range(6):
        new = torch.randint(-1, L, (M,), device="cuda", generator=g).int() if i % 3 else \
            torch.full((M,), i // 3 - 1, device="cuda").int()
        ids.copy_(new)
        want = step()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(p, e) for p, e in zip(out, want))
    q.q4gsw_device_error_check()
