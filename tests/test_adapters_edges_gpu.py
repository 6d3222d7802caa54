"""Adapters of many requests at the edges of what a call allows: plans that are shorter than the call's, terms that
pass fp16's range or nearly cancel the base product, plans of other batches."""
import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_adapters as oa
from test_adapters_gpu import check, close, head, make, q

pytestmark = pytest.mark.gpu


def c_call(name, *args):
    """The C function on the current stream, with tensors as their addresses: no check of Python's before it."""
    from bit_group_quantized_q4gsw_b200 import binding as b
    at = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    return getattr(b.library(), name)(*at, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("M", [12, 100, 600, 4100])
def test_a_plan_that_ends_before_the_calls_is_not_read_past_its_head(M):
    # the C calls have no size of the plan: the plan of one token, in a buffer of its own size, for M tokens.  The other
    # parts of a plan of M tokens would lie behind that buffer.
    m = q()
    N, K, gs, L, r = 64, 128, 32, 3, 8
    c = make(M, N, K, gs, L, r, np.arange(M) % L)
    blob, _, _, _, _, a, b = head(c)
    short = m.q4gsw_adapters_plan(torch.zeros(1, dtype=torch.int32, device="cuda"), L)
    assert 4 * short.numel() == 4 * (4 + 8 + 4 + 4 + 16 + 4)      # head, first, order, one tile, its rows, a pair
    x, d_y = cuda(c["x"]), cuda(c["d_y"])
    y, u, v = torch.zeros(M, N, device="cuda").half(), torch.full((M, r), 7.0, device="cuda"), torch.full((M, r), 7.0, device="cuda")
    d_x, d_a, d_b = torch.zeros(M, K, device="cuda").half(), torch.full((L, r, K), 5.0, device="cuda"), torch.full((L, N, r), 5.0, device="cuda")
    m.q4gsw_device_error_check()
    assert c_call("q4gsw_adapters_fwd", blob, N, K, gs, short, a, b, None, L, r, x, M, None, None, y, u) == 0
    with pytest.raises(m.Q4gswError, match="INDEX"):
        m.q4gsw_device_error_check()
    assert (u == 7).all()
    assert c_call("q4gsw_adapters_bwd", blob, N, K, gs, short, a, b, None, L, r, x, u, d_y, M, 0, v, d_x, d_a, d_b) == 0
    with pytest.raises(m.Q4gswError, match="INDEX"):
        m.q4gsw_device_error_check()
    assert (v == 7).all() and (d_a == 5).all() and (d_b == 5).all()
    m.q4gsw_adapters_fwd(*head(c), x)                              # the right plan still serves
    m.q4gsw_device_error_check()


def exact_case(M, f32s, L=3, N=136, K=128, r=16):
    """A base product of -8 times the first activation (forward) or gradient (backward), for every output, and adapters
    whose terms are picked by the next two: integers, exact in every sum."""
    m = q()
    codes = np.full((N, K), 8, np.uint8)
    codes[:, 0], codes[0, :] = 0, 0
    scales = np.ones((K // 32, N), np.float32 if f32s else np.float16)
    a, b = np.zeros((L, r, K), np.float16), np.zeros((L, N, r), np.float16)
    ids = (np.arange(M) % (L + 1) - 1).astype(np.int32)
    return m, m.q4gsw_prepack(cuda(codes), cuda(scales), 32), a, b, ids


@pytest.mark.parametrize("f32s", [False, True])
@pytest.mark.parametrize("M,gemm", [(M, None) for M in (1, 3, 8, 13, 16)] +
                         [(M, g) for M in (17, 40, 300, 513, 700, 1100) for g in (None, "ts", "ss1", "ss2")])
def test_a_term_that_leaves_the_range_of_fp16_or_cancels_the_base(M, gemm, f32s):
    # every sum is exact in fp32 and every output an fp16 value, so that outputs are equal: 60000 + 8000 - 20000 = 48000
    # (the residual with the term is 68000), and 40001 - 40000 = 1 (the term has 16 bits)
    m, blob, a, b, ids = exact_case(M, f32s)
    N, K, L, r = 136, 128, 3, 16
    with_adapter = torch.from_numpy(ids >= 0).cuda()[:, None]
    plan = m.q4gsw_adapters_plan(cuda(ids), L)
    m.q4gsw_debug_pin_routes(gemm=gemm) if gemm else m.q4gsw_debug_pin_routes()
    try:
        # forward: rank 0 has the activation 1, rank 1 the activation 2
        a[:, 0, 1], a[:, 1, 2] = 1, 1
        for base, first, second, res, want, alone in ((2500, 200, 0, 60000, 48000, 40000), (5000, 1000, 1, None, 1, -40000)):
            b[:, :, 0], b[:, :, 1] = 40, 1
            x = np.zeros((M, K), np.float16)
            x[:, 0], x[:, 1], x[:, 2] = base, first, second
            rest = None if res is None else torch.full((M, N), float(res), device="cuda").half()
            for y in (None, rest):       # and in the residual's own buffer
                y = m.q4gsw_adapters_fwd(blob, N, K, 32, plan, cuda(a), cuda(b), cuda(x), residual=rest, y=y, f32s=f32s)
                expect = torch.where(with_adapter, float(want), float(alone)).expand(M, N).clone()
                expect[:, 0] = torch.where(with_adapter[:, 0], want, alone) - 8 * (first + second)     # (row 0 of the weight is -8 everywhere)
                assert torch.equal(y.float(), expect.half().float()), (base, y[:, :3])
                if res is None:
                    break
        # backward: rank 0 has the gradient 1, rank 1 the gradient 2
        a[:], b[:] = 0, 0
        b[:, 1, 0], b[:, 2, 1] = 1, 1
        for base, first, second, want, alone in ((5000, 1000, 1, 1, -40000), (10000, 3000, 0, 40000, None)):
            a[:, 0, :], a[:, 1, :] = 40, 1
            d_y = np.zeros((M, N), np.float16)
            d_y[:, 0], d_y[:, 1], d_y[:, 2] = base, first, second
            d_x = m.q4gsw_adapters_bwd(blob, N, K, 32, plan, cuda(a), cuda(b), None, None, cuda(d_y), want_adapters=False, f32s=f32s)[0]
            got = d_x[ids >= 0][:, 1:]           # (column 0 of the weight is -8 in every row)
            assert torch.equal(got.float(), torch.full_like(got, want).float()), (base, d_x[:, :3])
            if alone is not None:
                got = d_x[ids < 0][:, 1:]
                assert torch.equal(got.float(), torch.full_like(got, alone).float())
    finally:
        m.q4gsw_debug_pin_routes()


@pytest.mark.parametrize("M,gemm", [(1, None), (5, None), (8, None), (16, None)] + [(M, g) for M in (17, 100, 600) for g in ("ts", "ss1", "ss2")])
def test_with_the_plan_of_another_batch_no_output_is_written(M, gemm):
    m = q()
    N, K, gs, L, r = 136, 256, 32, 3, 16
    c = make(M, N, K, gs, L, r, np.arange(M) % L)
    blob, _, _, _, plan, a, b = head(c)
    x, d_y, s = cuda(c["x"]), cuda(c["d_y"]), cuda(c["scale"])
    u = m.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, x, scale=s, save_u=True)[1]
    res = torch.randn(M, N, device="cuda").half()
    for other, its in ((M + 1, L), (M, L + 1)):
        wrong = m.q4gsw_adapters_plan(torch.zeros(other, dtype=torch.int32, device="cuda"), its,
                                      plan=torch.zeros(1 << 14, dtype=torch.int32, device="cuda"))
        m.q4gsw_device_error_check()
        m.q4gsw_debug_pin_routes(gemm=gemm) if gemm else m.q4gsw_debug_pin_routes()
        try:
            y = torch.full((M, N), 3.0, device="cuda").half()
            for residual, out, before in ((None, y, y.clone()), (res, y, y.clone()), (res, res, res.clone())):
                m.q4gsw_adapters_fwd(blob, N, K, gs, wrong, a, b, x, scale=s, residual=residual, y=out)
                with pytest.raises(m.Q4gswError, match="INDEX"):
                    m.q4gsw_device_error_check()
                assert torch.equal(out, before)
            d_x, v = torch.full((M, K), 3.0, device="cuda").half(), torch.full((M, r), 7.0, device="cuda")
            d_a, d_b = torch.full((L, r, K), 5.0, device="cuda"), torch.full((L, N, r), 5.0, device="cuda")
            m.q4gsw_adapters_bwd(blob, N, K, gs, wrong, a, b, x, u, d_y, scale=s, d_x=d_x, d_a=d_a, d_b=d_b, v=v)
            with pytest.raises(m.Q4gswError, match="INDEX"):
                m.q4gsw_device_error_check()
            assert (d_x == 3).all() and (v == 7).all() and (d_a == 5).all() and (d_b == 5).all()
        finally:
            m.q4gsw_debug_pin_routes()
    check(c, residual=res.cpu().numpy())                           # and the right plan still serves


@pytest.mark.parametrize("gemv", ["tma", "tma_xs"])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 11, 16])
def test_activations_and_plan_written_right_in_front_of_the_call(M, gemv):
    # the product reads x and the plan before it waits for the kernel in front: both are rewritten, in their own buffers, by
    # the kernels just before the call, many steps behind one another without a wait
    m = q()
    N, K, L, r = 520, 2048, 4, 16
    c = make(M, N, K, 32, L, r, np.arange(M) % L)
    blob, _, _, gs, _, a, b = head(c)
    g = torch.Generator(device="cuda").manual_seed(M)
    hs = [torch.empty(M, K, device="cuda").normal_(0, 1, generator=g).half() for _ in range(5)]
    ids = [torch.randint(-1, L, (M,), device="cuda", generator=g, dtype=torch.int32) for _ in range(7)]
    w = torch.ones(K, device="cuda").half()
    x, plan = torch.empty_like(hs[0]), torch.zeros_like(m.q4gsw_adapters_plan(ids[0], L))
    m.q4gsw_debug_pin_routes(gemv=gemv)
    try:
        want = {}
        for i in range(35):
            y = m.q4gsw_adapters_fwd(blob, N, K, gs, m.q4gsw_adapters_plan(ids[i % 7], L), a, b, m.q4gsw_norms_fwd(hs[i % 5], w_pre=w)[0])
            torch.cuda.synchronize()
            want[i] = y
        got = [torch.empty(M, N, device="cuda").half() for _ in range(35)]
        wrong = torch.zeros((), device="cuda", dtype=torch.int64)
        for _ in range(8):
            for i in range(35):
                if i % 2:
                    m.q4gsw_norms_fwd(hs[i % 5], w_pre=w, x=x)
                    m.q4gsw_adapters_plan(ids[i % 7], L, plan=plan)
                else:
                    m.q4gsw_adapters_plan(ids[i % 7], L, plan=plan)
                    m.q4gsw_norms_fwd(hs[i % 5], w_pre=w, x=x)
                m.q4gsw_adapters_fwd(blob, N, K, gs, plan, a, b, x, y=got[i])
            for i in range(35):
                wrong += (got[i] != want[i]).sum()
        assert wrong.item() == 0
    finally:
        m.q4gsw_debug_pin_routes()
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("M,L,N,K,r", [(1500, 1, 264, 320, 16), (3000, 2, 72, 128, 64), (2200, 3, 136, 64, 40)])
def test_accumulate_with_the_tokens_split_over_a_cluster(M, L, N, K, r):
    # few columns and many tokens of each adapter: the tokens' sums are added over a cluster's CTAs, then to the buffers
    m = q()
    c = make(M, N, K, 32, L, r, np.arange(M) * L // M)
    args, x, d_y, s = head(c), cuda(c["x"]), cuda(c["d_y"]), cuda(c["scale"])
    u = m.q4gsw_adapters_fwd(*args, x, scale=s, save_u=True)[1]
    _, d_a, d_b = m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s, want_x=False)
    want = oa.adapters_bwd(c["x"], u.cpu().numpy(), c["d_y"], c["w"], c["ids"], c["a"], c["b"], c["scale"])
    close(d_a, want[1], "d_a")
    close(d_b, want[2], "d_b")
    ga, gb = torch.randn_like(d_a), torch.randn_like(d_b)
    start = ga.clone(), gb.clone()
    for k in range(1, 4):          # micro-batches: the same sums once more each time
        m.q4gsw_adapters_bwd(*args, x, u, d_y, scale=s, want_x=False, d_a=ga, d_b=gb, accumulate=True)
        for got, first, grad in ((ga, start[0], d_a), (gb, start[1], d_b)):
            exact = first.double() + k * grad.double()
            assert ((got - exact).abs() <= k * 2.0 ** -24 * (first.abs().double() + k * grad.abs().double())).all()


def test_buffers_that_are_no_tensors_are_type_errors():
    m = q()
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="plan"):
        m.q4gsw_adapters_plan(ids, 2, plan=[0] * 64)
    x = torch.ones(2, 64, device="cuda").half()
    with pytest.raises(TypeError, match="workspace"):
        m.q4gsw_norms_bwd(x, d_x=x, w_pre=x[0], want_weights=True, workspace=b"0" * 4096)
    with pytest.raises(TypeError, match="workspace"):
        m.q4gsw_grad_norm(m.q4gsw_grad_set([torch.ones(200000, device="cuda")]), workspace=np.zeros(1 << 16, np.uint8))
