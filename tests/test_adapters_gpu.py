"""Adapters of many requests on the GPU: the plan, the forward and the backward
pass against the fp64 oracle, within bounds counted from the kernels' roundings."""
import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_adapters as oa
from oracle import q4gsw_layer as ol

pytestmark = pytest.mark.gpu


def q():
    import bit_group_quantized_q4gsw_b200 as m
    return m


def close(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == value.shape, (what, got.shape, value.shape)
    over = ~(np.abs(got - value) <= bound)
    if over.any():
        i = np.unravel_index(np.argmax(np.where(over, np.abs(got - value), 0)), got.shape)
        raise AssertionError(f"{what}: {over.sum()} of {over.size} outside; worst at {i}: got {got[i]!r} want {value[i]!r} "
                             f"bound {bound[i]!r} [{q().q4gsw_last_route()}]")


def make(M, N, K, gs, L, r, ids, f32s=False, seed=0, sigma=0.05):
    g = np.random.default_rng(seed + 1000 * M + N)
    codes = g.integers(0, 16, (N, K), dtype=np.uint8)
    scales = g.uniform(0.005, 0.02, (K // gs, N)).astype(np.float32 if f32s else np.float16)
    c = dict(M=M, N=N, K=K, gs=gs, L=L, r=r, f32s=f32s, ids=np.asarray(ids, np.int32), w=ol.dequant(codes, scales, gs),
             x=g.standard_normal((M, K)).astype(np.float16), d_y=(g.standard_normal((M, N)) * 0.05).astype(np.float16),
             a=(g.standard_normal((L, r, K)) * sigma).astype(np.float16),
             b=(g.standard_normal((L, N, r)) * sigma).astype(np.float16), scale=g.uniform(0.5, 2, L).astype(np.float32))
    c["blob"] = q().q4gsw_prepack(cuda(codes), cuda(scales), gs)
    c["plan"] = q().q4gsw_adapters_plan(cuda(c["ids"]), L)
    return c


def head(c):
    return c["blob"], c["N"], c["K"], c["gs"], c["plan"], cuda(c["a"]), cuda(c["b"])


def clean(ids, L):
    return np.where((ids >= 0) & (ids < L), ids, -1)


def runs(M, L, seed, none=True):
    """Ragged runs of tokens of one adapter, some without."""
    g = np.random.default_rng(seed)
    n = min(M, L + 3)
    cuts = np.sort(g.choice(M - 1, n - 1, replace=False)) + 1 if n > 1 else []
    return np.repeat(g.integers(-1 if none else 0, L, n), np.diff(np.concatenate([[0], cuts, [M]]).astype(int)))


# ---------------------------------------------------------------- plan
def read_plan(plan, M, L):
    p = plan.cpu().numpy()
    pad = lambda n: (n + 3) // 4 * 4      # noqa: E731
    slots = (M + 15 * min(L + 1, M)) // 16
    at = 4
    first = p[at:at + L + 2]
    at += pad(L + 2)
    order = p[at:at + M]
    at += pad(M)
    tile = p[at:at + slots]
    at += pad(slots)
    pairs = (slots + min(L + 1, M)) // 2
    return p[0], first, order, tile, p[at:at + 16 * slots].reshape(slots, 16), p[at + 16 * slots:at + 16 * slots + pairs]


@pytest.mark.parametrize("M,L", [(1, 1), (1, 1024), (2, 3), (16, 16), (17, 1), (33, 5), (512, 8), (1000, 1024), (1021, 40),
                                 (4096, 64), (100003, 257)])
@pytest.mark.parametrize("kind", ["random", "runs", "none", "one", "wild"])
def test_plan(M, L, kind):
    g = np.random.default_rng(M + L)
    ids = {"random": g.integers(-1, L, M), "runs": runs(M, L, M), "none": np.full(M, -1), "one": np.full(M, L - 1),
           "wild": g.integers(-3, L + 3, M)}[kind].astype(np.int32)
    m = q()
    m.q4gsw_device_error_check()
    plan = m.q4gsw_adapters_plan(cuda(ids), L)
    bad = ((ids < -1) | (ids >= L)).any()
    if bad:
        with pytest.raises(m.Q4gswError, match="INDEX"):
            m.q4gsw_device_error_check()
    m.q4gsw_device_error_check()
    tiles, first, order, tile, rows, pair = read_plan(plan, M, L)
    ids = clean(ids, L)
    group = np.where(ids < 0, L, ids)
    want = np.argsort(group, kind="stable")
    assert np.array_equal(order, want)
    counts = np.bincount(group, minlength=L + 1)
    assert np.array_equal(first, np.concatenate([[0], np.cumsum(counts)]))
    at = 0
    for a in np.nonzero(counts)[0]:
        n = -(-counts[a] // 16)
        assert (tile[at:at + n] == (a if a < L else -1)).all()
        flat = rows[at:at + n].ravel()
        assert np.array_equal(flat[:counts[a]], want[first[a]:first[a] + counts[a]]) and (flat[counts[a]:] == -1).all()
        at += n
    assert tiles == at and (tile[at:] == -2).all()
    starts = [i for i in range(at) if (i - int(np.argmax(tile[:at] == tile[i]))) % 2 == 0]      # every other tile of an adapter
    assert np.array_equal(pair[:len(starts)], starts) and (pair[len(starts):] == -1).all()


# ---------------------------------------------------------------- forward and backward
def check(c, bias=None, residual=None, scaled=True):
    m = q()
    s = c["scale"] if scaled else None
    ids = clean(c["ids"], c["L"])
    ts = cuda(s) if scaled else None
    y, u = m.q4gsw_adapters_fwd(*head(c), cuda(c["x"]), scale=ts, bias=None if bias is None else cuda(bias),
                                residual=None if residual is None else cuda(residual), save_u=True, f32s=c["f32s"])
    want_y, want_u = oa.adapters_fwd(c["x"], c["w"], ids, c["a"], c["b"], s, bias, residual)
    close(u, want_u, "u")
    close(y, want_y, "y")
    assert not u[cuda(ids) < 0].any()
    d_x, d_a, d_b = m.q4gsw_adapters_bwd(*head(c), cuda(c["x"]), u, cuda(c["d_y"]), scale=ts, f32s=c["f32s"])
    want = oa.adapters_bwd(c["x"], u.cpu().numpy(), c["d_y"], c["w"], ids, c["a"], c["b"], s)
    close(d_x, want[0], "d_x")
    close(d_a, want[1], "d_a")
    close(d_b, want[2], "d_b")
    m.q4gsw_device_error_check()
    return y, u, d_x, d_a, d_b


CASES = [
    # M, N, K, gs, L, r, f32s
    (1, 8, 64, 16, 1, 8, False), (1, 2048, 2048, 32, 4, 16, False), (2, 72, 448, 64, 5, 24, True),
    (5, 264, 1088, 16, 3, 32, True), (9, 40, 320, 32, 16, 40, False), (16, 520, 4096, 128, 32, 16, False),
    (16, 136, 576, 64, 16, 64, False), (17, 8, 64, 64, 2, 48, False), (33, 136, 192, 32, 7, 56, True),
    (64, 1000, 1024, 128, 1, 64, False), (200, 328, 2048, 32, 9, 8, False), (256, 64, 4096, 512, 3, 16, False),
    (508, 1032, 512, 16, 8, 16, False), (513, 72, 320, 64, 40, 24, False), (700, 264, 576, 32, 4, 40, True),
    (1030, 520, 1024, 128, 6, 64, False), (1200, 200, 256, 32, 1, 32, False),
]


@pytest.mark.parametrize("M,N,K,gs,L,r,f32s", CASES)
def test_ragged_runs(M, N, K, gs, L, r, f32s):
    check(make(M, N, K, gs, L, r, runs(M, L, M + r), f32s))


@pytest.mark.parametrize("M,N,K,gs,L,r,f32s", CASES[1::2])
def test_tokens_in_no_order_with_bias_and_residual(M, N, K, gs, L, r, f32s):
    g = np.random.default_rng(M)
    c = make(M, N, K, gs, L, r, g.integers(-1, L, M), f32s)
    check(c, bias=g.standard_normal(N).astype(np.float16), residual=g.standard_normal((M, N)).astype(np.float16),
          scaled=False)


@pytest.mark.parametrize("r", range(8, 72, 8))
@pytest.mark.parametrize("M", [3, 50])
def test_every_rank(r, M):
    check(make(M, 152, 192, 32, 4, r, runs(M, 4, r)))


def test_no_token_has_an_adapter():
    c = make(40, 136, 256, 32, 3, 16, np.full(40, -1))
    res = np.random.default_rng(1).standard_normal((40, 136)).astype(np.float16)
    y, u, d_x, d_a, d_b = check(c, residual=res)
    m = q()
    assert not u.any() and not d_a.any() and not d_b.any()
    assert torch.equal(y, m.q4gsw_linear_act_fwd(c["blob"], 136, 256, 32, cuda(c["x"]), residual=cuda(res)))


def test_one_adapter_for_all_equals_the_single_adapter_operator():
    c = make(100, 256, 512, 32, 1, 16, np.zeros(100))
    y = check(c, scaled=False)[0].float()
    one = q().q4gsw_adapter_fwd(c["blob"], 256, 512, 32, cuda(c["a"][0]), cuda(c["b"][0]), cuda(c["x"]))
    assert (y - one).abs().max() <= 2 ** -9 * one.abs().max()      # fp16 outputs of the same sums


@pytest.mark.parametrize("M", [5, 40, 300])
def test_integers_are_exact(M):
    # small integers: every product and sum is exact, the outputs too
    g = np.random.default_rng(M)
    N, K, L, r = 72, 128, 4, 16
    codes = g.integers(7, 10, (N, K), dtype=np.uint8)
    w = codes.astype(np.float64) - 8
    ids = g.integers(-1, L, M).astype(np.int32)
    x = g.integers(-1, 2, (M, K)).astype(np.float16)
    a, b = g.integers(-1, 2, (L, r, K)).astype(np.float16), g.integers(-1, 2, (L, N, r)).astype(np.float16)
    d_y = g.integers(-1, 2, (M, N)).astype(np.float16)
    scale = np.array([1, 2, -1, 0.5], np.float32)
    m = q()
    blob = m.q4gsw_prepack(cuda(codes), cuda(np.ones((K // 32, N), np.float16)), 32)
    plan = m.q4gsw_adapters_plan(cuda(ids), L)
    args = (blob, N, K, 32, plan, cuda(a), cuda(b))
    y, u = m.q4gsw_adapters_fwd(*args, cuda(x), scale=cuda(scale), save_u=True)
    (wy, _), (wu, _) = oa.adapters_fwd(x, w, ids, a, b, scale)
    assert np.array_equal(u.cpu().numpy(), wu) and np.array_equal(y.cpu().numpy(), wy)
    d_x, d_a, d_b = m.q4gsw_adapters_bwd(*args, cuda(x), u, cuda(d_y), scale=cuda(scale))
    (wx, _), (wa, _), (wb, _) = oa.adapters_bwd(x, wu, d_y, w, ids, a, b, scale)
    assert np.array_equal(d_x.cpu().numpy(), wx)
    assert np.array_equal(d_a.cpu().numpy(), wa) and np.array_equal(d_b.cpu().numpy(), wb)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_the_intermediate_keeps_its_range(size):
    # u and v far outside fp16's range: factors bring the products back
    c = make(20, 64, 128, 32, 2, 16, np.arange(20) % 3 - 1)
    u = torch.randn(20, 16, device="cuda") * size
    u[cuda(c["ids"]) < 0] = 0
    s = np.array([1 / size, 2 / size], np.float32)
    _, d_a, d_b = q().q4gsw_adapters_bwd(*head(c), cuda(c["x"]), u, cuda(c["d_y"]), scale=cuda(s), want_x=False)
    want = oa.adapters_bwd(c["x"], u.cpu().numpy(), c["d_y"], c["w"], c["ids"], c["a"], c["b"], s)
    close(d_b, want[2], "d_b")
    close(d_a, want[1], "d_a")
    s = np.array([size, -size], np.float32)       # v = s d_y B, and v A into an fp16 d_x where that holds it
    if size < 1:
        d_x, d_a, _ = q().q4gsw_adapters_bwd(*head(c), cuda(c["x"]), u, cuda(c["d_y"]), scale=cuda(s))
        want = oa.adapters_bwd(c["x"], u.cpu().numpy(), c["d_y"], c["w"], c["ids"], c["a"], c["b"], s)
        close(d_x, want[0], "d_x")
        close(d_a, want[1], "d_a")


def test_a_token_that_is_not_finite_stays_alone():
    c = make(48, 136, 256, 32, 3, 16, np.arange(48) % 4 - 1)
    base = q().q4gsw_adapters_fwd(*head(c), cuda(c["x"]), scale=cuda(c["scale"]))
    for bad, value in ((5, np.nan), (6, np.inf), (7, -np.inf)):
        c["x"][bad, 17] = value
    y = q().q4gsw_adapters_fwd(*head(c), cuda(c["x"]), scale=cuda(c["scale"]))
    rest = [m for m in range(48) if m not in (5, 6, 7)]
    assert torch.equal(y[rest], base[rest]) and not torch.isfinite(y[5]).any()
    # an adapter that is not finite reaches its own tokens alone; one without tokens nobody
    c = make(48, 136, 256, 32, 4, 16, np.arange(48) % 3)
    base = q().q4gsw_adapters_fwd(*head(c), cuda(c["x"]))
    grads = q().q4gsw_adapters_bwd(*head(c), cuda(c["x"]), torch.ones(48, 16, device="cuda"), cuda(c["d_y"]))
    c["a"][3], c["b"][3] = np.nan, np.inf
    assert torch.equal(q().q4gsw_adapters_fwd(*head(c), cuda(c["x"])), base)
    again = q().q4gsw_adapters_bwd(*head(c), cuda(c["x"]), torch.ones(48, 16, device="cuda"), cuda(c["d_y"]))
    assert all(torch.equal(v, w) for v, w in zip(grads, again))
    c["a"][1] = np.nan
    y = q().q4gsw_adapters_fwd(*head(c), cuda(c["x"]))
    rest = [m for m in range(48) if m % 3 != 1]
    assert torch.equal(y[rest], base[rest]) and torch.isnan(y[1::3]).all()


def test_accumulate_and_parts_of_the_backward_pass():
    m = q()
    c = make(70, 136, 256, 32, 4, 24, runs(70, 3, 2))
    args = head(c)
    x, d_y, s = cuda(c["x"]), cuda(c["d_y"]), cuda(c["scale"])
    u = m.q4gsw_adapters_fwd(*args, x, scale=s, save_u=True)[1]
    d_x, d_a, d_b = m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s)
    only = m.q4gsw_adapters_bwd(*args, None, None, d_y, scale=s, want_adapters=False)
    assert torch.equal(only[0], d_x) and only[1] is None and only[2] is None
    only = m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s, want_x=False)
    assert only[0] is None and torch.equal(only[1], d_a) and torch.equal(only[2], d_b)
    ga, gb = torch.randn_like(d_a), torch.randn_like(d_b)
    a0, b0 = ga.clone(), gb.clone()
    m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s, want_x=False, d_a=ga, d_b=gb, accumulate=True)
    for got, start, grad in ((ga, a0, d_a), (gb, b0, d_b)):
        want = start.double() + grad.double()
        assert ((got - want).abs() <= 2.0 ** -23 * (want.abs() + grad.abs().double())).all()
    assert torch.equal(ga[3], a0[3]) and torch.equal(gb[3], b0[3])       # no tokens: left alone
    with pytest.raises(ValueError, match="accumulate"):
        m.q4gsw_adapters_bwd(*args, x, u, d_y, accumulate=True)


def test_residual_in_place_and_buffers():
    m = q()
    c = make(30, 136, 256, 32, 3, 16, runs(30, 3, 4))
    res = torch.randn(30, 136, device="cuda").half()
    want = m.q4gsw_adapters_fwd(*head(c), cuda(c["x"]), scale=cuda(c["scale"]), residual=res)
    again = m.q4gsw_adapters_fwd(*head(c), cuda(c["x"]), scale=cuda(c["scale"]), residual=res, y=res)
    assert again is res and torch.equal(res, want)


def test_empty_batch():
    m = q()
    c = make(4, 64, 128, 32, 2, 8, [0, 1, -1, 0])
    plan = m.q4gsw_adapters_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    a, b = cuda(c["a"]), cuda(c["b"])
    x, d_y, u = (torch.empty(0, n, device="cuda") for n in (128, 64, 8))
    y = m.q4gsw_adapters_fwd(c["blob"], 64, 128, 32, plan, a, b, x.half())
    assert y.shape == (0, 64)
    d_x, d_a, d_b = m.q4gsw_adapters_bwd(c["blob"], 64, 128, 32, plan, a, b, x.half(), u, d_y.half())
    assert d_x.shape == (0, 128) and not d_a.any() and not d_b.any()


def test_repeats_streams_and_graphs():
    m = q()
    c = make(300, 264, 512, 32, 5, 16, np.random.default_rng(3).integers(-1, 5, 300))
    args, x, d_y, s = head(c), cuda(c["x"]), cuda(c["d_y"]), cuda(c["scale"])

    def both(plan):
        a = (*args[:4], plan, *args[5:])
        y, u = m.q4gsw_adapters_fwd(*a, x, scale=s, save_u=True)
        return (y, u, *m.q4gsw_adapters_bwd(*a, x, u, d_y, scale=s))

    ids = cuda(c["ids"])
    want = both(args[4])
    for _ in range(20):
        assert all(torch.equal(v, w) for v, w in zip(both(args[4]), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(m.q4gsw_adapters_plan(ids, 5))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(v, w) for v, w in zip(got, want))
    # plan, forward and backward in one captured graph, replayed for other ids and activations
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(m.q4gsw_adapters_plan(ids, 5))
    graph.replay()
    assert all(torch.equal(v, w) for v, w in zip(got, want))
    ids.copy_(torch.randint(-1, 5, (300,), device="cuda", dtype=torch.int32))
    x.copy_(torch.randn_like(x))
    graph.replay()
    again = both(m.q4gsw_adapters_plan(ids, 5))
    assert all(torch.equal(v, w) for v, w in zip(got, again))
    m.q4gsw_device_error_check()


def test_offsets_past_2_31_elements():
    # 1024 adapters of [40960, 64]: the last lies behind 2.6e9 elements
    m = q()
    L, N, K, r, M = 1024, 40960, 64, 64, 20
    g = np.random.default_rng(0)
    codes = g.integers(0, 16, (N, K), dtype=np.uint8)
    scales = g.uniform(0.005, 0.02, (2, N)).astype(np.float16)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), 32)
    ids = np.array([1023, 0, -1, 1022] * 5, np.int32)
    a, b = torch.zeros(L, r, K, device="cuda").half(), torch.zeros(L, N, r, device="cuda", dtype=torch.float16)
    keep = [0, 1022, 1023]
    for i in keep:
        a[i], b[i] = torch.randn(r, K, device="cuda") * 0.1, torch.randn(N, r, device="cuda") * 0.1
    x, d_y = g.standard_normal((M, K)).astype(np.float16), (g.standard_normal((M, N)) * 0.05).astype(np.float16)
    plan = m.q4gsw_adapters_plan(cuda(ids), L)
    y, u = m.q4gsw_adapters_fwd(blob, N, K, 32, plan, a, b, cuda(x), save_u=True)
    d_x, d_a, d_b = m.q4gsw_adapters_bwd(blob, N, K, 32, plan, a, b, cuda(x), u, cuda(d_y))
    small = np.array([2, 0, -1, 1] * 5)
    w, sa, sb = ol.dequant(codes, scales, 32), a[keep].cpu().numpy(), b[keep].cpu().numpy()
    want_y, want_u = oa.adapters_fwd(x, w, small, sa, sb)
    close(u, want_u, "u")
    close(y, want_y, "y")
    want = oa.adapters_bwd(x, u.cpu().numpy(), d_y, w, small, sa, sb)
    close(d_x, want[0], "d_x")
    close(d_a[keep], want[1], "d_a")
    close(d_b[keep], want[2], "d_b")
    assert not d_b[1:1022].any() and not d_a[1:1022].any()


def test_python_checks():
    m = q()
    c = make(20, 64, 128, 32, 2, 8, np.zeros(20))
    blob, N, K, gs, plan, a, b = head(c)
    x = cuda(c["x"])
    for bad, what in (((blob, N, K, gs, plan, a[:, :, :64].contiguous(), b, x), "a must have"),
                      ((blob, N, K, gs, plan, a, b[:1], x), "b must have"), ((blob, N, K, gs, plan[:8], a, b, x), "plan holds"),
                      ((blob, N, K, gs, plan, a[0], b, x), "3 dims"), ((blob[:100], N, K, gs, plan, a, b, x), "packed holds")):
        with pytest.raises(ValueError, match=what):
            m.q4gsw_adapters_fwd(*bad)
    with pytest.raises(TypeError, match="plan"):
        m.q4gsw_adapters_fwd(blob, N, K, gs, plan.float(), a, b, x)
    with pytest.raises(ValueError, match="scale"):
        m.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, x, scale=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError, match="u must be"):
        m.q4gsw_adapters_bwd(blob, N, K, gs, plan, a, b, x, torch.zeros(20, 8, device="cuda").half(), cuda(c["d_y"]))


@pytest.mark.parametrize("M", [1, 8, 16, 40, 600])
def test_steps_back_to_back_reuse_their_buffers(M):
    # a norm writes x, the projection reads it before the low-rank kernels in front of it are done: 200 steps on
    # the same buffers without a wait give what each gives alone
    m = q()
    K, N, L, r = 2048, 256, 3, 16
    c = make(M, N, K, 32, L, r, np.arange(M) % (L + 1) - 1)
    args, s = head(c), cuda(c["scale"])
    g = torch.Generator(device="cuda").manual_seed(M)
    hs = [torch.empty(M, K, device="cuda").normal_(0, 1, generator=g).half() for _ in range(8)]
    w = torch.empty(K, device="cuda").normal_(1, 0.1, generator=g).half()
    d_y = torch.empty(M, N, device="cuda").normal_(0, 0.1, generator=g).half()
    want = []
    for h in hs:
        x, _ = m.q4gsw_norms_fwd(h, w_pre=w)
        torch.cuda.synchronize()
        y, u = m.q4gsw_adapters_fwd(*args, x, scale=s, save_u=True)
        torch.cuda.synchronize()
        want.append((y, u, *m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s)))
        torch.cuda.synchronize()
    x, y, u = torch.empty_like(hs[0]), torch.empty(M, N, device="cuda").half(), torch.empty(M, r, device="cuda")
    v, d_x = torch.empty_like(u), torch.empty_like(x)
    d_a, d_b = torch.empty(L, r, K, device="cuda"), torch.empty(L, N, r, device="cuda")
    wrong = torch.zeros((), device="cuda", dtype=torch.int64)
    for i in range(200):
        m.q4gsw_norms_fwd(hs[i % 8], w_pre=w, x=x)
        m.q4gsw_adapters_fwd(*args, x, scale=s, y=y, u=u)
        m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s, d_x=d_x, d_a=d_a, d_b=d_b, v=v)
        if i % 3 == 0:      # (a comparison is a kernel in between: most steps follow each other at once)
            for got, ref in zip((y, u, d_x, d_a, d_b), want[i % 8]):
                wrong += (got != ref).sum()
    assert wrong.item() == 0
    m.q4gsw_device_error_check()


def test_a_plan_of_another_batch_computes_nothing():
    m = q()
    for M, other in ((40, 41), (40, 39), (600, 599), (600, 602)):
        c = make(M, 64, 128, 32, 3, 8, np.arange(M) % 3)
        blob, N, K, gs, plan, a, b = head(c)
        x, u = cuda(c["x"]), torch.full((M, 8), 7.0, device="cuda")
        big = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
        wrong = m.q4gsw_adapters_plan(torch.zeros(other, dtype=torch.int32, device="cuda"), 3, plan=big)
        y = torch.full((M, 64), 3.0, device="cuda").half()
        m.q4gsw_device_error_check()
        m.q4gsw_adapters_fwd(blob, N, K, gs, wrong, a, b, x, y=y, u=u)
        with pytest.raises(m.Q4gswError, match="INDEX"):
            m.q4gsw_device_error_check()
        assert (u == 7).all()
        d_a, d_b = torch.full((3, 8, K), 5.0, device="cuda"), torch.full((3, N, 8), 5.0, device="cuda")
        v = u.clone()
        m.q4gsw_adapters_bwd(blob, N, K, gs, wrong, a, b, x, u, cuda(c["d_y"]), d_a=d_a, d_b=d_b, v=v)
        with pytest.raises(m.Q4gswError, match="INDEX"):
            m.q4gsw_device_error_check()
        assert (d_a == 5).all() and (d_b == 5).all() and (v == 7).all()
        m.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, x)
        m.q4gsw_device_error_check()


@pytest.mark.parametrize("gemm", ["ts", "ss1", "ss2"])
@pytest.mark.parametrize("M", [40, 600])
def test_every_gemm_route_behind_the_low_rank_kernels(M, gemm):
    m = q()
    c = make(M, 264, 320, 32, 3, 16, runs(M, 3, M))
    m.q4gsw_debug_pin_routes(gemm=gemm)
    try:
        check(c, residual=np.random.default_rng(2).standard_normal((M, 264)).astype(np.float16))
    finally:
        m.q4gsw_debug_pin_routes()


@pytest.mark.parametrize("M,N,K,L,r,kind", [(3000, 72, 192, 700, 8, "random"), (5000, 136, 128, 1, 64, "one"), (4100, 264, 64, 2, 24, "runs"),
                                            (2049, 200, 128, 130, 32, "random"), (1500, 64, 4160, 5, 40, "runs")])
def test_many_tiles(M, N, K, L, r, kind):
    # the ring kernels: pairs with one and two tiles, one and two adapters to a CTA, token splits of the gradients
    g = np.random.default_rng(M)
    ids = {"random": g.integers(-1, L, M), "one": np.zeros(M), "runs": runs(M, L, M)}[kind]
    check(make(M, N, K, 32, L, r, ids), residual=g.standard_normal((M, N)).astype(np.float16))


def test_two_streams_share_a_plan_and_the_adapters():
    m = q()
    c = make(700, 264, 512, 32, 4, 32, runs(700, 4, 1))
    args, s = head(c), cuda(c["scale"])
    xs = [torch.randn(700, 512, device="cuda").half() for _ in range(2)]
    d_y = cuda(c["d_y"])

    def both(x):
        y, u = m.q4gsw_adapters_fwd(*args, x, scale=s, save_u=True)
        return (y, u, *m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s))

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for k, side in enumerate(streams):
            with torch.cuda.stream(side):
                got[k].append(both(xs[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(v, w) for v, w in zip(run, want[k]))


@pytest.mark.parametrize("M,N,K,gs,r,f32s", [(9, 4160, 4096, 64, 8, False), (16, 4096, 4160, 64, 16, True), (12, 14336, 2432, 128, 16, False),
                                               (6, 1032, 8192, 128, 16, False), (8, 4096, 4096, 32, 8, True), (1, 264, 4160, 64, 16, False)])
def test_low_rank_kernels_beside_the_product(M, N, K, gs, r, f32s):
    # up to 16 tokens of a large projection: the low-rank CTAs run while the product's stream the weight; the
    # residual in place, many steps behind one another on the same buffers
    m = q()
    L = 6
    c = make(M, N, K, gs, L, r, np.arange(M) % (L + 1) - 1, f32s)
    g = np.random.default_rng(M)
    res = g.standard_normal((M, N)).astype(np.float16)
    check(c, bias=g.standard_normal(N).astype(np.float16), residual=res)
    args, s = head(c), cuda(c["scale"])
    xs = [torch.randn(M, K, device="cuda").half() for _ in range(4)]
    want = []
    for x in xs:
        y = m.q4gsw_adapters_fwd(*args, x, scale=s, residual=cuda(res), f32s=f32s)
        torch.cuda.synchronize()
        want.append(y)
    first, u = cuda(res), torch.empty(M, r, device="cuda")
    buf = [torch.empty_like(first) for _ in range(2)]
    wrong = torch.zeros((), device="cuda", dtype=torch.int64)
    for i in range(200):
        y = buf[i % 2]
        m.q4gsw_norms_fwd(first, residual_scale=1.0, h_out=y)                # the residual's buffer, which the call overwrites
        m.q4gsw_adapters_fwd(*args, xs[i % 4], scale=s, residual=y, y=y, u=u, f32s=f32s)
        if i % 5 == 0:
            wrong += (y != want[i % 4]).sum()
    assert wrong.item() == 0
    m.q4gsw_device_error_check()


def test_outputs_over_inputs_that_are_read_later_are_refused():
    m = q()
    c = make(20, 128, 128, 32, 2, 8, runs(20, 2, 0))
    args, x, d_y = head(c), cuda(c["x"]), cuda(c["d_y"])
    before = x.clone()
    with pytest.raises(ValueError, match="y must not be x's buffer"):
        m.q4gsw_adapters_fwd(*args, x, residual=x, y=x)
    y, u = m.q4gsw_adapters_fwd(*args, x, residual=x, save_u=True)
    for kw in (dict(d_x=d_y), dict(d_x=x), dict(v=u)):
        with pytest.raises(ValueError, match="must not be"):
            m.q4gsw_adapters_bwd(*args, x, u, d_y, **kw)
    assert torch.equal(x, before)
    close(m.q4gsw_adapters_bwd(*args, x, u, d_y, d_x=x, want_adapters=False)[0],      # x is not read without d_a and d_b
          oa.adapters_bwd(before.cpu().numpy(), u.cpu().numpy(), c["d_y"], c["w"], clean(c["ids"], 2), c["a"], c["b"], None)[0], "d_x")
