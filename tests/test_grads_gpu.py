"""The norm and the clip of a list of gradients on the GPU against fp64, and the
operators of an adapter's training step together."""
import math

import numpy as np
import pytest
import torch

from oracle import q4gsw_adapters as oa

pytestmark = pytest.mark.gpu


def q():
    import bit_group_quantized_q4gsw_b200 as m
    return m


def lists(sizes, halves, seed=0, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.empty(n, device="cuda").normal_(0, sigma, generator=g)).to(torch.float16 if h else torch.float32)
            for n, h in zip(sizes, halves)]


def host(t):
    return t.detach().cpu().numpy()


def check(grads, outs=None, max_norm=1.0, inv=1.0):
    m = q()
    before = [host(g) for g in grads]
    n, b = oa.grad_norm(before, inv)
    s = m.q4gsw_grad_set(grads, outs)
    norm = m.q4gsw_grad_norm(s, inv_scale=inv)
    assert abs(norm.item() - n) <= b, (norm.item(), n)
    assert all(np.array_equal(host(g), v) for g, v in zip(grads, before))
    again = m.q4gsw_grad_clip(s, max_norm, inv_scale=inv)
    assert torch.equal(again, norm)
    to = grads if outs is None else outs
    clipped = {h: oa.grad_clip(before, max_norm, inv, h) for h in (False, True)}
    for i, t in enumerate(to):
        want, bound = clipped[t.dtype is torch.float16][i]
        assert (np.abs(host(t).astype(np.float64) - want) <= bound).all(), i
    if outs is not None:
        assert all(np.array_equal(host(g), v) for g, v in zip(grads, before))
    return norm


@pytest.mark.parametrize("sizes", [[1], [7], [8192], [8193, 0, 5], [16384, 8191, 3, 100000], [0, 0, 9], [3000000, 17, 40000]])
@pytest.mark.parametrize("half", [0, 1, 2])
def test_sizes_and_types(sizes, half):
    halves = [half == 1 or (half == 2 and i % 2) for i in range(len(sizes))]
    check(lists(sizes, halves))
    check(lists(sizes, halves, 1), [torch.zeros(n, device="cuda") for n in sizes], max_norm=0.25, inv=0.5)
    check(lists(sizes, halves, 2), [torch.zeros(n, device="cuda", dtype=torch.float16) for n in sizes], max_norm=3.0)


def test_many_tensors_and_pieces():
    g = np.random.default_rng(1)
    sizes = [int(v) for v in g.integers(1, 3000, 1500)]
    check(lists(sizes, [i % 3 == 0 for i in range(1500)]))
    big = lists([40_000_003, 9], [0, 1])          # more pieces than CTAs
    check(big, max_norm=100.0)


@pytest.mark.parametrize("shift", range(1, 8))
@pytest.mark.parametrize("half", [False, True])
def test_views_at_any_element(shift, half):
    flat = lists([70000], [half], shift)[0]
    out = torch.full((70010,), 7.0, device="cuda", dtype=flat.dtype)
    views = [flat[shift:shift + 20001], flat[shift + 20001:shift + 20001 + 30000]]
    outs = [out[shift + 2:shift + 2 + 20001], out[shift + 2 + 20001:shift + 2 + 50001]]
    check(views, outs)
    assert (out[:shift + 2] == 7).all() and (out[shift + 50003:] == 7).all()
    check([v.clone() for v in views])


def test_values_whose_squares_leave_fp32():
    for size in (1e-38, 1e-25, 1e25, 1e36):
        check(lists([5000, 33], [0, 0], sigma=size), max_norm=size, inv=1.0)
    check(lists([4], [0], sigma=1e-44), max_norm=1.0)          # subnormal gradients


def test_a_set_keeps_the_storages_it_has_addresses_of():
    m = q()
    g = lists([3000], [0])
    s, old = m.q4gsw_grad_set(g), g[0].detach()
    where, copy = old.data_ptr(), old.clone()
    del old
    g[0].data = torch.zeros(3000, device="cuda")          # another storage; the set has the old one
    torch.cuda.synchronize()
    fresh = [torch.zeros(3000, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() != where for t in fresh)
    want = float(copy.double().pow(2).sum().sqrt())
    assert abs(float(m.q4gsw_grad_norm(s)) - want) <= want * 2 ** -23


def test_factor_of_one_leaves_the_gradients_alone():
    m = q()
    g = lists([1000, 50], [0, 1])
    want = [t.clone() for t in g]
    m.q4gsw_grad_clip(m.q4gsw_grad_set(g), 1e9)
    assert all(torch.equal(v, w) for v, w in zip(g, want))
    m.q4gsw_grad_clip(m.q4gsw_grad_set(g), math.inf, inv_scale=0.5)
    assert all(torch.equal(v, w * 0.5) for v, w in zip(g, want))
    outs = [torch.zeros(1000, device="cuda"), torch.zeros(50, device="cuda")]
    m.q4gsw_grad_clip(m.q4gsw_grad_set(want, outs), 1e9)
    assert all(torch.equal(v, w.float()) for v, w in zip(outs, want))


def test_gradients_that_are_not_finite():
    m = q()
    for bad in (math.inf, -math.inf, math.nan):
        g = lists([100, 3000], [0, 0])
        g[1][77] = bad
        s = m.q4gsw_grad_set(g)
        n = m.q4gsw_grad_norm(s).item()
        assert math.isnan(n) if math.isnan(bad) else n == math.inf
        m.q4gsw_grad_clip(s, 1.0)
        if math.isnan(bad):
            assert all(torch.isnan(t).all() for t in g)
        else:
            assert torch.isnan(g[1][77]) and not g[0].any() and not g[1][:77].any()     # 0 times infinity, else 0


def test_zero_gradients():
    g = [torch.zeros(5000, device="cuda")]
    assert check(g).item() == 0 and not g[0].any()


def test_refusals():
    m = q()
    a, b = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    for grads, outs, what in (([a, a], None, "overlap"), ([a[:60], a[50:]], None, "overlap"), ([a, b], [b, a], "overlap"),
                              ([a], [a[1:]], "elements"), ([a], [a.view(torch.float16)[:100]], "overlap"),
                              ([a, b], [a], "outs for"), ([a[::2]], None, "contiguous")):
        with pytest.raises(ValueError, match=what):
            m.q4gsw_grad_set(grads, outs)
    with pytest.raises(TypeError, match="float32 or float16"):
        m.q4gsw_grad_set([a.double()])
    s = m.q4gsw_grad_set([a], [b])
    for v in (0.0, -1.0, math.nan):
        with pytest.raises(m.Q4gswError, match="SHAPE"):
            m.q4gsw_grad_clip(s, v)


def test_repeats_streams_and_graphs():
    m = q()
    g = lists([100000, 3333, 8192 * 7], [0, 1, 0])
    outs = [torch.zeros(t.numel(), device="cuda") for t in g]
    s = m.q4gsw_grad_set(g, outs)
    n = m.q4gsw_grad_clip(s, 1.0)
    want = [o.clone() for o in outs]
    for _ in range(20):
        assert torch.equal(m.q4gsw_grad_clip(s, 1.0), n) and all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2 = m.q4gsw_grad_clip(s, 1.0)
    [t.mul_(3) for t in g]
    graph.replay()
    torch.cuda.synchronize()
    n3, bound = oa.grad_norm([host(t) for t in g])
    assert abs(n2.item() - n3) <= bound
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n4 = m.q4gsw_grad_clip(s, 1.0)
    side.synchronize()
    assert torch.equal(n4, n2)


# ---------------------------------------------------------------- a step of them together
def test_a_training_step_of_a_feed_forward_block():
    """Pre norm, up projection with each token's adapter, post norm onto the stream and the next pre norm; back
    again, and the clip of every gradient: against torch's derivatives in fp64."""
    m = q()
    M, D, L, r, gs = 96, 256, 3, 16, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, k=1.0: torch.empty(*s, device="cuda").normal_(0, k, generator=g)      # noqa: E731
    codes = torch.randint(0, 16, (D, D), device="cuda", dtype=torch.uint8, generator=g)
    scales = torch.empty(D // gs, D, device="cuda").uniform_(0.005, 0.02, generator=g).half()
    blob = m.q4gsw_prepack(codes, scales, gs)
    ids = torch.randint(-1, L, (M,), device="cuda", dtype=torch.int32, generator=g)
    h, a, b = n(M, D).half(), n(L, r, D, k=0.05).half(), n(L, D, r, k=0.05).half()
    s = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    w1, w2, w3 = (n(D, k=0.2).half() for _ in range(3))
    d_x, d_h = n(M, D, k=0.1).half(), n(M, D, k=0.1).half()

    plan = m.q4gsw_adapters_plan(ids, L)
    x1, _ = m.q4gsw_norms_fwd(h, w_pre=w1, weight_offset=1.0)
    y, u = m.q4gsw_adapters_fwd(blob, D, D, gs, plan, a, b, x1, scale=s, save_u=True)
    x2, h2 = m.q4gsw_norms_fwd(h, block=y, w_post=w2, w_pre=w3, weight_offset=1.0)
    back = m.q4gsw_norms_bwd(h2, d_x=d_x, d_h=d_h, block=y, w_post=w2, w_pre=w3, weight_offset=1.0, want_weights=True)
    d_x1, d_a, d_b = m.q4gsw_adapters_bwd(blob, D, D, gs, plan, a, b, x1, u, back.block, scale=s)
    first = m.q4gsw_norms_bwd(h, d_x=d_x1, d_h=back.residual, w_pre=w1, weight_offset=1.0, want_weights=True)
    mine = dict(h=first.residual, w1=first.w_pre, a=d_a, b=d_b, w2=back.w_post, w3=back.w_pre)
    want = {k: v.clone() for k, v in mine.items()}
    grads = [mine[k] for k in ("w1", "a", "b", "w2", "w3")]
    norm = m.q4gsw_grad_clip(m.q4gsw_grad_set(grads), 0.1)
    m.q4gsw_device_error_check()

    leaf = {k: v.double().requires_grad_() for k, v in dict(h=h, w1=w1, a=a, b=b, w2=w2, w3=w3).items()}
    w = (codes.double() - 8) * torch.repeat_interleave(scales.double(), gs, 0).t()
    rms = lambda v, k: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * (1 + leaf[k])      # noqa: E731
    e1 = rms(leaf["h"], "w1")
    at = ids.clamp_min(0).long()
    low = torch.einsum("mk,mrk->mr", e1, leaf["a"][at])
    low = torch.einsum("mr,mnr->mn", low, leaf["b"][at]) * (s.double()[at] * (ids >= 0)).unsqueeze(1)
    e2 = leaf["h"] + rms(e1 @ w.t() + low, "w2")
    ((rms(e2, "w3") * d_x.double()).sum() + (e2 * d_h.double()).sum()).backward()
    # fp16 steps of the chain's five tensors and of the weights, 2^-11 each, through at most
    # a norm's gain: 2^-8 of the 2-norm of each result
    for k, v in leaf.items():
        got = want[k].double()
        assert (got - v.grad).norm() <= 2.0 ** -8 * v.grad.norm(), k
    total = math.sqrt(sum(float((want[k].double() ** 2).sum()) for k in ("w1", "a", "b", "w2", "w3")))
    assert abs(norm.item() - total) <= 1e-6 * total
    for k in ("w1", "a", "b", "w2", "w3"):
        assert torch.allclose(mine[k], want[k] * min(1.0, 0.1 / (total + 1e-6)), rtol=1e-6, atol=0)


@pytest.mark.parametrize("n", [1024 * 55, 1024 * 56, 1024 * 57, 1024 * 64, 1024 * 65 + 1])
def test_around_the_length_where_one_launch_becomes_two(n):
    # a record more than the tensor's own may stand in the table (the largest offset it may start at)
    m = q()
    g = lists([n - 5000, 5000], [0, 1], n)
    check(g, [torch.zeros(n - 5000, device="cuda"), torch.zeros(5000, device="cuda")], max_norm=2.0)
    s = m.q4gsw_grad_set(g)
    a = m.q4gsw_grad_norm(s)
    one = "launches=1" in m.q4gsw_last_route()
    assert one == (s.table_bytes <= 64 * 32)
    ws = torch.empty(8192, dtype=torch.uint8, device="cuda")
    assert torch.equal(m.q4gsw_grad_norm(s, workspace=ws), a)
