"""The gated feed-forward block and the projection with an epilogue against
the fp64 oracle, within bounds counted from the kernels' roundings."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_group_quantized_q4gsw_b200 import workloads as wl
from helpers import cuda
from oracle import q4gsw_layer as ol

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def q():
    import bit_group_quantized_q4gsw_b200 as m
    return m


def weight(N, K, gs, f32s, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.uniform(0.005, 0.02, (K // gs, N))
    return codes, scales.astype(np.float32 if f32s else np.float16)


def close(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == value.shape, (what, got.shape, value.shape)
    over = np.abs(got - value) > bound
    if over.any():
        i = np.unravel_index(np.argmax(np.abs(got - value) / bound), got.shape)
        raise AssertionError(f"{what}: {over.sum()} outside; worst at {i}: got {got[i]!r} want {value[i]!r} "
                             f"bound {bound[i]!r} [{q().q4gsw_last_route()}]")


# every route: GEMV of 1..8 and 9..16 tokens (one and several splits), the two
# GEMMs with and without split-K; F and K off the tile sizes; every group size
GATED = [
    (1, 8, 64, 16, False), (1, 8192, 2048, 32, False), (2, 72, 448, 64, True), (5, 264, 1088, 16, True),
    (8, 520, 4096, 4096, False), (9, 40, 320, 32, False), (16, 1544, 1024, 256, True), (16, 8, 14336, 128, False),
    (17, 8, 64, 64, False), (33, 136, 192, 32, True), (64, 1000, 1024, 128, False), (200, 328, 2048, 32, False),
    (256, 64, 8192, 512, False), (508, 1024, 512, 16, False), (513, 72, 320, 64, False), (700, 264, 576, 32, True),
    (1030, 520, 1024, 128, False),
]


@pytest.mark.parametrize("M,F,K,gs,f32s", GATED)
def test_gated_forward_and_backward(M, F, K, gs, f32s):
    m = q()
    cg, sg = weight(F, K, gs, f32s, 1)
    cu, su = weight(F, K, gs, f32s, 2)
    wg, wu = ol.dequant(cg, sg, gs), ol.dequant(cu, su, gs)
    blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    rng = np.random.default_rng(M + F)
    x = rng.standard_normal((M, K)).astype(np.float16)
    d_h = (rng.standard_normal((M, F)) * 0.05).astype(np.float16)
    kind = "silu" if (M + F // 8) % 2 else "gelu_tanh"
    want_h, want_gu = ol.gated_fwd(x, wg, wu, kind)
    h, gu = m.q4gsw_gated_fwd(blob, F, K, gs, cuda(x), act=kind, save_gu=True, f32s=f32s)
    close(h, want_h, "h")
    close(gu, want_gu, "gu")
    only = m.q4gsw_gated_fwd(blob, F, K, gs, cuda(x), act=kind, f32s=f32s)
    assert torch.equal(only, h)                       # the same bits whether g and u are saved or not
    d_x, d_gu = m.q4gsw_gated_bwd(blob, F, K, gs, gu, cuda(d_h), act=kind, f32s=f32s)
    want_dx, want_dgu = ol.gated_bwd(gu.cpu().numpy(), d_h, wg, wu, kind)
    close(d_gu, want_dgu, "d_gu")
    close(d_x, want_dx, "d_x")
    into = gu.clone()                                 # in place over the saved pairs
    d_x2, same = m.q4gsw_gated_bwd(blob, F, K, gs, into, cuda(d_h), act=kind, d_gu=into, f32s=f32s)
    assert same is into and torch.equal(into, d_gu) and torch.equal(d_x2, d_x)
    m.q4gsw_device_error_check()


def test_prepack_gated_is_the_packing_of_the_interleaved_rows():
    m = q()
    for f32s in (False, True):
        cg, sg = weight(72, 192, 64, f32s, 3)
        cu, su = weight(72, 192, 64, f32s, 4)
        codes = np.stack([cg, cu], 1).reshape(144, 192)
        scales = np.stack([sg, su], 2).reshape(3, 144)
        a = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), 64)
        assert torch.equal(a, m.q4gsw_prepack(cuda(codes), cuda(scales), 64))
    bad = cu.copy()
    bad[5, 7] = 16
    with pytest.raises(m.Q4gswError) as e:
        m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(bad), cuda(su), 64)
    assert e.value.status_name == "Q4GSW_ERR_CODE_RANGE"


LINEAR = [
    (1, 8, 64, 16, False, "none", False, True), (1, 2048, 8192, 32, False, "none", False, True),
    (3, 200, 448, 64, True, "gelu_tanh", True, False), (8, 1032, 2048, 128, False, "silu", True, True),
    (12, 72, 14336, 128, False, "none", True, True), (16, 520, 1088, 64, True, "silu", False, False),
    (17, 8, 64, 16, False, "gelu_tanh", True, True), (77, 264, 448, 16, False, "none", False, False),
    (130, 1048, 1024, 32, True, "gelu_tanh", True, False), (508, 2048, 1024, 32, False, "none", True, True),
    (512, 136, 4096, 256, False, "silu", True, True), (600, 200, 192, 64, False, "gelu_tanh", True, True),
    (1030, 392, 1024, 128, True, "none", True, True), (2600, 4104, 64, 64, False, "gelu_tanh", True, False),
]


@pytest.mark.parametrize("M,N,K,gs,f32s,kind,with_bias,with_res", LINEAR)
def test_linear_act_forward_and_backward(M, N, K, gs, f32s, kind, with_bias, with_res):
    m = q()
    codes, scales = weight(N, K, gs, f32s, 5)
    w = ol.dequant(codes, scales, gs)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    rng = np.random.default_rng(M + N)
    x = rng.standard_normal((M, K)).astype(np.float16)
    bias = rng.standard_normal(N).astype(np.float16) if with_bias else None
    res = rng.standard_normal((M, N)).astype(np.float16) if with_res else None
    d_y = (rng.standard_normal((M, N)) * 0.05).astype(np.float16)
    dev = lambda a: None if a is None else cuda(a)   # noqa: E731
    want_y, want_z = ol.linear_act_fwd(x, w, kind, bias, res)
    y, z = m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), bias=dev(bias), act=kind, residual=dev(res), save_z=True,
                                  f32s=f32s)
    close(y, want_y, "y")
    close(z, want_z, "z")
    if with_res:                                      # the residual stream updated in place
        stream = dev(res)
        out = m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), bias=dev(bias), act=kind, residual=stream, y=stream,
                                     f32s=f32s)
        assert out is stream and torch.equal(stream, y)
    zz = z if kind != "none" else None
    d_x, d_z, d_b = m.q4gsw_linear_act_bwd(blob, N, K, gs, cuda(d_y), z=zz, act=kind, want_bias=True, f32s=f32s)
    want_dx, want_dz, want_db = ol.linear_act_bwd(z.cpu().numpy(), d_y, w, kind)
    close(d_x, want_dx, "d_x")
    close(d_b, want_db, "d_bias")
    if kind == "none":
        assert d_z is None
    else:
        close(d_z, want_dz, "d_z")
        again = cuda(d_y)                             # in place over d_y, no bias gradient: the same bits
        d_x2, d_z2, none = m.q4gsw_linear_act_bwd(blob, N, K, gs, again, z=zz, act=kind, d_z=again, f32s=f32s)
        assert none is None and torch.equal(d_z2, d_z) and torch.equal(d_x2, d_x)
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("M", [1, 7, 16, 40, 300, 600])
def test_integer_inputs_give_exact_results(M):
    """Integer activations and power-of-two scales: every product and sum is exact in fp32, so y is the
    fp16 rounding of the true value, bit for bit."""
    m = q()
    N, K, gs = 264, 448, 64
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = np.exp2(rng.integers(-3, 2, (K // gs, N))).astype(np.float16)
    w = ol.dequant(codes, scales, gs)
    x = rng.integers(-2, 3, (M, K)).astype(np.float16)
    bias = rng.integers(-8, 9, N).astype(np.float16)
    res = rng.integers(-64, 65, (M, N)).astype(np.float16)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    y, z = m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), bias=cuda(bias), residual=cuda(res), save_z=True)
    exact = x.astype(np.float64) @ w.T + bias
    assert np.array_equal(z.cpu().numpy(), exact.astype(np.float16))
    assert np.array_equal(y.cpu().numpy(), (exact + res).astype(np.float16))
    d = rng.integers(-2, 3, (M, N)).astype(np.float16)
    d_x, _, d_b = m.q4gsw_linear_act_bwd(blob, N, K, gs, cuda(d), want_bias=True)
    assert np.array_equal(d_x.cpu().numpy(), (d.astype(np.float64) @ w).astype(np.float16))
    assert np.array_equal(d_b.cpu().numpy(), d.astype(np.float64).sum(0).astype(np.float32))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gradient_against_differences_of_the_forward(kind):
    """<d_h, h(x + s v) - h(x - s v)> / 2 s from the fp64 forward against <d_x, v> from the kernels."""
    m = q()
    M, F, K, gs = 24, 136, 128, 32
    cg, sg = weight(F, K, gs, False, 6)
    cu, su = weight(F, K, gs, False, 7)
    wg, wu = ol.dequant(cg, sg, gs), ol.dequant(cu, su, gs)
    rng = np.random.default_rng(8)
    x = rng.standard_normal((M, K)).astype(np.float16)
    d_h = (rng.standard_normal((M, F)) * 0.1).astype(np.float16)
    blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    _, gu = m.q4gsw_gated_fwd(blob, F, K, gs, cuda(x), act=kind, save_gu=True)
    d_x, _ = m.q4gsw_gated_bwd(blob, F, K, gs, gu, cuda(d_h), act=kind)
    d_x = d_x.cpu().numpy().astype(np.float64)
    # d_x differs from the true gradient by its bound and by the rounding of the saved g and u
    _, (want_gu, b_gu) = ol.gated_fwd(x, wg, wu, kind)
    (_, b_dx), _ = ol.gated_bwd(want_gu, d_h, wg, wu, kind)
    d_abs = np.abs(d_h.astype(np.float64))
    moved = b_gu.reshape(M, F, 2)
    shift = d_abs * (moved[:, :, 1] * 1.13 + 1.2 * moved[:, :, 0] * (np.abs(want_gu[:, 1::2]) + 1))
    for _ in range(5):
        v, s = rng.standard_normal(x.shape), 1e-4
        f = lambda t: (ol.gated_fwd(x + t * v, wg, wu, kind)[0][0] * d_h).sum()   # noqa: E731
        diff = (f(s) - f(-s)) / (2 * s)
        tol = (b_dx * np.abs(v)).sum() + (shift @ (np.abs(wg) + np.abs(wu)) * np.abs(v)).sum() + 1e-6
        assert abs(diff - (d_x * v).sum()) <= tol


def test_values_at_the_ends_of_the_fp16_range():
    """Activations far from zero: the exponential overflows or vanishes, the results stay the limits."""
    m = q()
    F, K, gs = 8, 64, 64
    one = np.full((F, K), 8, np.uint8)
    one[:, 0] = 9                                      # w = 1 at column 0, zero elsewhere
    ones = np.ones((1, F), np.float16)
    blob = m.q4gsw_prepack_gated(cuda(one), cuda(ones), cuda(one), cuda(ones), gs)
    vals = np.array([-60000, -300, -90, -20, -1e-3, 0, 1e-3, 20, 90, 250], np.float16)
    x = np.zeros((len(vals), K), np.float16)
    x[:, 0] = vals
    v = vals.astype(np.float64)
    for kind in ("silu", "gelu_tanh"):
        h, gu = m.q4gsw_gated_fwd(blob, F, K, gs, cuda(x), act=kind, save_gu=True)
        with np.errstate(over="ignore"):
            want = ol.act(v, kind) * v
        got = h.cpu().numpy()[:, 0].astype(np.float64)
        assert np.abs(got - want).max() <= 2.0 ** -10 * np.abs(want).max() and np.isfinite(got).all()
        d_x, d_gu = m.q4gsw_gated_bwd(blob, F, K, gs, gu, torch.full((len(vals), F), 0.5, dtype=torch.float16).cuda(),
                                      act=kind)
        assert torch.isfinite(d_gu).all()
        with np.errstate(over="ignore"):
            want_g = 0.5 * v * ol.slope(v, kind)
        assert np.abs(d_gu.cpu().numpy()[:, 0] - want_g).max() <= 2.0 ** -10 * np.abs(want_g).max()


def test_a_nan_token_stays_in_its_row():
    m = q()
    for M in (3, 40, 600):
        F, K, gs = 72, 128, 32
        cg, sg = weight(F, K, gs, False, 9)
        blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cg), cuda(sg), gs)
        x = torch.randn(M, K, device="cuda").half()
        clean = m.q4gsw_gated_fwd(blob, F, K, gs, x)
        x[1, 5] = float("nan")
        h = m.q4gsw_gated_fwd(blob, F, K, gs, x)
        keep = [i for i in range(M) if i != 1]
        assert torch.isnan(h[1]).all() and torch.equal(h[keep], clean[keep])


def test_rows_behind_the_batch_are_left_alone():
    m = q()
    for M in (1, 5, 16, 40, 130, 520):
        F, K, gs = 72, 192, 64
        cg, sg = weight(F, K, gs, False, 10)
        blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cg), cuda(sg), gs)
        x = torch.randn(M, K, device="cuda").half()
        h = torch.full((M + 3, F), 7.0, dtype=torch.float16, device="cuda")
        gu = torch.full((M + 3, 2 * F), 7.0, dtype=torch.float16, device="cuda")
        m.q4gsw_gated_fwd(blob, F, K, gs, x, h=h[:M], gu=gu[:M])
        d_x = torch.full((M + 3, K), 7.0, dtype=torch.float16, device="cuda")
        d_gu = torch.full((M + 3, 2 * F), 7.0, dtype=torch.float16, device="cuda")
        m.q4gsw_gated_bwd(blob, F, K, gs, gu[:M], h[:M], d_gu=d_gu[:M], d_x=d_x[:M])
        for t in (h, gu, d_x, d_gu):
            assert (t[M:] == 7.0).all() and (t[:M] != 7.0).any()


def test_empty_batches():
    m = q()
    codes, scales = weight(64, 128, 32, False, 11)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), 32)
    x = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    assert m.q4gsw_linear_act_fwd(blob, 64, 128, 32, x).shape == (0, 64)
    d = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    d_x, _, d_b = m.q4gsw_linear_act_bwd(blob, 64, 128, 32, d, want_bias=True)
    assert d_x.shape == (0, 128) and (d_b == 0).all()


@pytest.mark.parametrize("M", [1, 12, 100, 512, 1024])
def test_repeats_streams_and_graphs_give_the_same_bits(M):
    m = q()
    F, K, gs = 1032, 1024, 32
    cg, sg = weight(F, K, gs, False, 12)
    cu, su = weight(F, K, gs, False, 13)
    blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    x = torch.randn(M, K, device="cuda").half()
    d_h = torch.randn(M, F, device="cuda").half() * 0.01

    def step():
        h, gu = m.q4gsw_gated_fwd(blob, F, K, gs, x, save_gu=True)
        return (h, gu) + m.q4gsw_gated_bwd(blob, F, K, gs, gu, d_h)

    first = step()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(step(), first))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:                                  # several calls at once
        with torch.cuda.stream(s):
            outs.append([step() for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for r in o for a, b in zip(r, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x.copy_(torch.randn(M, K, device="cuda").half())   # new inputs in the captured buffers
    for _ in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    m.q4gsw_device_error_check()


def test_python_checks_of_shapes():
    m = q()
    codes, scales = weight(128, 128, 32, False, 14)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), 32)
    x = torch.zeros(4, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="x must have shape"):
        m.q4gsw_linear_act_fwd(blob, 64, 64, 32, x)
    with pytest.raises(ValueError, match="packed holds"):
        m.q4gsw_linear_act_fwd(blob, 256, 128, 32, x)
    with pytest.raises(ValueError, match="residual"):
        m.q4gsw_linear_act_fwd(blob, 128, 128, 32, x, residual=torch.zeros(4, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError, match="bias"):
        m.q4gsw_linear_act_fwd(blob, 128, 128, 32, x, bias=torch.zeros(128, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        m.q4gsw_linear_act_fwd(blob, 128, 128, 32, torch.zeros(128, 4, dtype=torch.float16, device="cuda").t())
    with pytest.raises(ValueError, match="act must be"):
        m.q4gsw_gated_fwd(blob, 64, 128, 32, x, act="none")
    with pytest.raises(ValueError, match="z is required"):
        m.q4gsw_linear_act_bwd(blob, 128, 128, 32, x, act="silu")
    with pytest.raises(m.Q4gswError) as e:
        m.q4gsw_gated_fwd(blob, 60, 128, 32, x)
    assert e.value.status_name == "Q4GSW_ERR_ALIGN"


@pytest.mark.parametrize("gemm", ["ts", "ss1", "ss2"])
@pytest.mark.parametrize("M", [40, 300, 700])
def test_both_gemm_routes_agree_with_the_oracle(gemm, M):
    m = q()
    F, K, gs = 200, 1088, 64
    cg, sg = weight(F, K, gs, False, 15)
    cu, su = weight(F, K, gs, False, 16)
    wg, wu = ol.dequant(cg, sg, gs), ol.dequant(cu, su, gs)
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)).astype(np.float16)
    d_h = (rng.standard_normal((M, F)) * 0.05).astype(np.float16)
    blob = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    m.q4gsw_debug_pin_routes(gemm=gemm)
    try:
        h, gu = m.q4gsw_gated_fwd(blob, F, K, gs, cuda(x), save_gu=True)
        d_x, d_gu = m.q4gsw_gated_bwd(blob, F, K, gs, gu, cuda(d_h))
    finally:
        m.q4gsw_debug_pin_routes()
    want_h, want_gu = ol.gated_fwd(x, wg, wu, "silu")
    close(h, want_h, "h")
    close(gu, want_gu, "gu")
    want_dx, want_dgu = ol.gated_bwd(gu.cpu().numpy(), d_h, wg, wu, "silu")
    close(d_x, want_dx, "d_x")
    close(d_gu, want_dgu, "d_gu")


# few input features: no split, so that every output goes out by tensor stores; tiles of 256 columns and 128 or
# 256 tokens that end inside the output, one sub-tile and two, with and without room for both at once
@pytest.mark.parametrize("gemm", ["ss1", "ss2"])
@pytest.mark.parametrize("M,N,K", [(17, 8, 64), (128, 72, 192), (129, 264, 448), (257, 520, 128), (640, 1048, 192)])
def test_whole_sums_of_the_shared_memory_gemm(gemm, M, N, K):
    m = q()
    gs = 32
    codes, scales = weight(N, K, gs, False, 31)
    w = ol.dequant(codes, scales, gs)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    rng = np.random.default_rng(M + N)
    x = rng.standard_normal((M, K)).astype(np.float16)
    bias = rng.standard_normal(N).astype(np.float16)
    res = rng.standard_normal((M, N)).astype(np.float16)
    d_y = (rng.standard_normal((M, N)) * 0.05).astype(np.float16)
    m.q4gsw_debug_pin_routes(gemm=gemm)
    try:
        for kind, b, r, save in (("gelu_tanh", bias, res, True), ("silu", None, res, False), ("none", bias, None, False),
                                 ("silu", bias, None, True)):
            y, z = (torch.full((M + 2, N), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
            if r is not None:
                y[:M] = cuda(r)                       # the residual stream updated in place
            m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), bias=None if b is None else cuda(b), act=kind,
                                   residual=None if r is None else y[:M], y=y[:M], z=z[:M] if save else None)
            assert "out=epi" in m.q4gsw_last_route() and m.q4gsw_last_route().split("grid=")[1].split()[0].endswith("x1")
            want_y, want_z = ol.linear_act_fwd(x, w, kind, b, r)
            close(y[:M], want_y, f"y {kind}")
            if save:
                close(z[:M], want_z, f"z {kind}")
            assert (y[M:] == 7.0).all() and (z[M if save else 0:] == 7.0).all()
        F = N // 16 * 8
        cg, sg = weight(F, K, gs, False, 32)
        cu, su = weight(F, K, gs, False, 33)
        gated = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs) if F else None
        if F:
            wg, wu = ol.dequant(cg, sg, gs), ol.dequant(cu, su, gs)
            h, gu = m.q4gsw_gated_fwd(gated, F, K, gs, cuda(x), act="gelu_tanh", save_gu=True)
            want_h, want_gu = ol.gated_fwd(x, wg, wu, "gelu_tanh")
            close(h, want_h, "h")
            close(gu, want_gu, "gu")
            assert torch.equal(h, m.q4gsw_gated_fwd(gated, F, K, gs, cuda(x), act="gelu_tanh"))
        d_x, _, _ = m.q4gsw_linear_act_bwd(blob, N, K, gs, cuda(d_y))
        close(d_x, ol.linear_act_bwd(None, d_y, w, "none")[0], "d_x")
    finally:
        m.q4gsw_debug_pin_routes()
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("gemm,M", [("ss1", 520), ("ss2", 1040)])
def test_tiles_left_over_by_whole_waves(gemm, M):
    """30 x 5 output tiles on 148 SMs: two of them in a second launch that splits the contraction."""
    m = q()
    N, K, gs = 7680, 2048, 128
    codes, scales = weight(N, K, gs, False, 34)
    w = ol.dequant(codes, scales, gs)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)).astype(np.float16)
    res = rng.standard_normal((M, N)).astype(np.float16)
    want_y, want_z = ol.linear_act_fwd(x, w, "silu", None, res)
    m.q4gsw_debug_pin_routes(gemm=gemm)
    try:
        y = cuda(res)
        _, z = m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), act="silu", residual=y, y=y, save_z=True)
        if torch.cuda.get_device_properties(0).multi_processor_count == 148:
            assert "launches=2" in m.q4gsw_last_route() and "rest_splits=" in m.q4gsw_last_route()
        close(y, want_y, "y")
        close(z, want_z, "z")
        g = torch.cuda.CUDAGraph()
        y2 = torch.empty_like(y)
        xs, rs = cuda(x), cuda(res)
        side = torch.cuda.Stream()
        with torch.cuda.graph(g, stream=side):
            m.q4gsw_linear_act_fwd(blob, N, K, gs, xs, act="silu", residual=rs, y=y2)
        for _ in range(3):
            y2.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y2, y)
    finally:
        m.q4gsw_debug_pin_routes()
    m.q4gsw_device_error_check()


def test_workload_shapes_of_the_1b_layer_run_as_one_block():
    """norm-free feed-forward half of a layer: gated block, down projection onto the residual, and back."""
    m = q()
    up, down = wl.adapter()[0], wl.adapter()[1]
    M, K, F, gs = 64, up.K, up.N, up.group_size
    cg, sg = weight(F, K, gs, False, 17)
    cu, su = weight(F, K, gs, False, 18)
    cd, sd = weight(down.N, down.K, gs, False, 19)
    wg, wu, wd = ol.dequant(cg, sg, gs), ol.dequant(cu, su, gs), ol.dequant(cd, sd, gs)
    rng = np.random.default_rng(20)
    x = rng.standard_normal((M, K)).astype(np.float16)
    d_y = (rng.standard_normal((M, K)) * 1e-2).astype(np.float16)
    gated = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    dn = m.q4gsw_prepack(cuda(cd), cuda(sd), gs)
    xd = cuda(x)
    h, gu = m.q4gsw_gated_fwd(gated, F, K, gs, xd, save_gu=True)
    y = m.q4gsw_linear_act_fwd(dn, K, F, gs, h, residual=xd)
    d_h, _, _ = m.q4gsw_linear_act_bwd(dn, K, F, gs, cuda(d_y))
    d_x, _ = m.q4gsw_gated_bwd(gated, F, K, gs, gu, d_h)
    close(y, ol.linear_act_fwd(h.cpu().numpy(), wd, "none", residual=x)[0], "y")
    close(d_h, ol.linear_act_bwd(None, d_y, wd, "none")[0], "d_h")
    close(d_x, ol.gated_bwd(gu.cpu().numpy(), d_h.cpu().numpy(), wg, wu, "silu")[0], "d_x")
    m.q4gsw_device_error_check()


FIRST_CALL_CAPTURED = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import bit_group_quantized_q4gsw_b200 as q
torch.manual_seed(0)
F, K, gs, V, k = 264, 512, 32, 1000, 8
def w(N):
    return (torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda"),
            (torch.rand(K // gs, N, device="cuda") * 0.01).half())
gate, up, proj = w(F), w(F), w(F)
gated = q.q4gsw_prepack_gated(*gate, *up, gs)
blob = q.q4gsw_prepack(*proj, gs)
for M in (1, 12, 100, 600):
    x, d = torch.randn(M, K, device="cuda").half(), torch.randn(M, F, device="cuda").half() * 0.01
    z = torch.randn(M, V, device="cuda")
    idx = torch.randint(0, V, (M, k), device="cuda").int()
    t, dl = torch.randn(M, k, device="cuda"), torch.ones(M, device="cuda")
    bias = torch.randn(F, device="cuda").half()
    def step():
        h, gu = q.q4gsw_gated_fwd(gated, F, K, gs, x, save_gu=True)
        y, zz = q.q4gsw_linear_act_fwd(blob, F, K, gs, x, bias=bias, act="silu", residual=h, save_z=True)
        out = q.q4gsw_gated_bwd(gated, F, K, gs, gu, d) + q.q4gsw_linear_act_bwd(blob, F, K, gs, d, z=zz, act="silu",
                                                                               want_bias=True)
        loss, lse, g = q.q4gsw_distill_step(z, idx, t, dl, 2.0)
        return (h, y) + out + (loss, lse, g, q.q4gsw_distill_bwd(z, lse, idx, t, dl, 2.0)) + \
            q.q4gsw_distill_fwd(z, idx, t, 2.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):          # the first call of every kernel of this batch size
        captured = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step())), M
q.q4gsw_device_error_check()
print("first calls captured ok")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "first calls captured ok" in r.stdout


def test_a_kernel_before_and_after_on_the_same_stream():
    """The calls overlap their start with the kernel before them (programmatic dependent launch): inputs written,
    and outputs read, by neighbouring kernels of the stream are seen in order."""
    m = q()
    F, K, gs = 1024, 1024, 32
    cg, sg = weight(F, K, gs, False, 21)
    cu, su = weight(F, K, gs, False, 22)
    cd, sd = weight(K, F, gs, False, 23)
    gated = m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs)
    down = m.q4gsw_prepack(cuda(cd), cuda(sd), 32)
    for M in (1, 16, 100, 700):
        x0 = torch.randn(M, K, device="cuda").half()
        want = x0.clone()
        for _ in range(3):          # waits between the calls
            h = m.q4gsw_gated_fwd(gated, F, K, gs, want)
            torch.cuda.synchronize()
            want = m.q4gsw_linear_act_fwd(down, K, F, gs, h, residual=want)
            torch.cuda.synchronize()
        for _ in range(5):          # none, and the residual stream updated in place
            x = x0.clone()
            for _ in range(3):
                m.q4gsw_linear_act_fwd(down, K, F, gs, m.q4gsw_gated_fwd(gated, F, K, gs, x), residual=x, y=x)
            # bit patterns: the third layer's products pass the fp16 range, and a NaN equals nothing
            assert torch.equal(x.view(torch.int16), want.view(torch.int16))
        # the same with one layer a call, whose values are all finite
        one = m.q4gsw_linear_act_fwd(down, K, F, gs, m.q4gsw_gated_fwd(gated, F, K, gs, x0), residual=x0)
        torch.cuda.synchronize()
        assert torch.isfinite(one).all()
        for _ in range(20):
            x = x0.clone()
            m.q4gsw_linear_act_fwd(down, K, F, gs, m.q4gsw_gated_fwd(gated, F, K, gs, x), residual=x, y=x)
            assert torch.equal(x, one)
