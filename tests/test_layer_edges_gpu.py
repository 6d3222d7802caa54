"""Edges of the layer operators: saved infinities, the rules that choose a kernel, random shapes."""
import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_layer as ol
from test_layer_gpu import close, q, weight

pytestmark = pytest.mark.gpu


def test_saved_values_beyond_the_fp16_range_give_the_limits_of_the_gradient():
    """g, u and z past the fp16 range are saved as infinities; act and its slope have limits there, and a token
    whose own gradient is zero stays at zero."""
    m = q()
    F, K, gs = 16, 64, 64
    blob = m.q4gsw_prepack(cuda(np.full((F, K), 9, np.uint8)), cuda(np.ones((1, F), np.float16)), gs)
    gated = m.q4gsw_prepack_gated(*(cuda(a) for a in 2 * (np.full((F, K), 9, np.uint8), np.ones((1, F), np.float16))), gs)
    inf = np.inf
    z = np.array([inf, -inf, 3.0, np.nan], np.float16)[:, None].repeat(F, 1)
    for kind in ("silu", "gelu_tanh"):
        for M in (4, 20):
            zz = np.concatenate([z, np.zeros((M - 4, F), np.float16)])
            d_y = np.full((M, F), 0.5, np.float16)
            _, d_z, d_b = m.q4gsw_linear_act_bwd(blob, F, K, gs, cuda(d_y), z=cuda(zz), act=kind, want_bias=True)
            d_z = d_z.cpu().numpy()
            assert (d_z[0] == 0.5).all() and (d_z[1] == 0).all() and np.isfinite(d_z[2]).all() and np.isnan(d_z[3]).all()
            # pairs (g, u): the slope's and the value's limits, an infinite u, and no gradient at all
            gu = np.zeros((M, 2 * F), np.float16)
            pairs = [(inf, 2), (-inf, 2), (-inf, inf), (inf, inf), (1, -inf), (-inf, -inf), (np.nan, 1), (1, np.nan)]
            gu[0, :16], gu[1, :16] = np.ravel(pairs), np.ravel(pairs)
            d_h = np.full((M, F), 0.5, np.float16)
            d_h[1] = 0
            _, d_gu = m.q4gsw_gated_bwd(gated, F, K, gs, cuda(gu), cuda(d_h), act=kind)
            d_g, d_u = d_gu.cpu().numpy()[:2, 0::2], d_gu.cpu().numpy()[:2, 1::2]
            assert np.array_equal(d_g[0, :6], np.array([1, 0, 0, inf, -inf, 0], np.float16))
            assert np.array_equal(d_u[0, [0, 1, 2, 3, 5]], np.array([inf, 0, 0, inf, 0], np.float16))
            assert np.isfinite(d_u[0, 4])
            assert (d_g[1, :6] == 0).all() and (d_u[1, :6] == 0).all()
            assert np.isnan(d_g[0, 6:8]).all() and np.isnan(d_u[0, 6])


def launches(route):
    """The kernels of a call: every part of a route counts its own."""
    return sum(int(w.split("=")[1]) for w in route.split() if w.startswith("launches="))


def test_routes_count_every_launch():
    m = q()
    N, K, gs = 72, 128, 32
    blob = m.q4gsw_prepack(*(cuda(a) for a in weight(N, K, gs, False, 41)), gs)
    for M in (3, 40):
        d = torch.randn(M, N, device="cuda").half()
        z = torch.randn(M, N, device="cuda").half()
        for want, f in ((1, lambda: m.q4gsw_linear_act_bwd(blob, N, K, gs, d)),
                        (2, lambda: m.q4gsw_linear_act_bwd(blob, N, K, gs, d, want_bias=True)),
                        (2, lambda: m.q4gsw_linear_act_bwd(blob, N, K, gs, d, z=z, act="silu"))):
            f()
            assert launches(m.q4gsw_last_route()) == want, m.q4gsw_last_route()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def block(F, K, gs, f32s, seed):
    """(packed, gate, up) of a gated block."""
    m = q()
    cg, sg = weight(F, K, gs, f32s, seed)
    cu, su = weight(F, K, gs, f32s, seed + 1)
    return (m.q4gsw_prepack_gated(cuda(cg), cuda(sg), cuda(cu), cuda(su), gs), ol.dequant(cg, sg, gs),
            ol.dequant(cu, su, gs))


@pytest.mark.parametrize("M", [256, 257, 500, 512])
def test_the_kernel_that_fits_one_wave(M):
    """257 to 512 tokens on about as many 256 x 256 tiles as there are SMs, which the tensor-memory kernel's
    smaller tiles take two waves for: the shared-memory kernel, unpinned; up to 256 tokens the other one."""
    m = q()
    F, K, gs = 128 * (sms() // 2) - 24, 192, 64
    packed, wg, wu = block(F, K, gs, False, 42)
    x = np.random.default_rng(M).standard_normal((M, K)).astype(np.float16)
    h, gu = m.q4gsw_gated_fwd(packed, F, K, gs, cuda(x), save_gu=True)
    assert ("tcgen05_gemm_fwd" if M > 256 else "tcgen05_ts_gemm_fwd") in m.q4gsw_last_route()
    want_h, want_gu = ol.gated_fwd(x, wg, wu, "silu")
    close(h, want_h, "h")
    close(gu, want_gu, "gu")
    # the input gradient of a projection whose input is as wide
    codes, scales = weight(K, 2 * F // 64 * 64, gs, False, 44)
    back = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    d_y = (np.random.default_rng(M + 1).standard_normal((M, K)) * 0.05).astype(np.float16)
    d_x, _, _ = m.q4gsw_linear_act_bwd(back, K, codes.shape[1], gs, cuda(d_y))
    assert ("tcgen05_gemm_bwd" if M > 256 else "tcgen05_ts_gemm_bwd") in m.q4gsw_last_route()
    close(d_x, ol.linear_act_bwd(None, d_y, ol.dequant(codes, scales, gs), "none")[0], "d_x")
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("f32s", [False, True])
@pytest.mark.parametrize("gemm,M", [("ss1", 520), ("ss2", 1040)])
def test_left_over_tiles_of_gated_outputs_and_of_gradients(gemm, M, f32s):
    """Five rows of tiles, of which one to five tiles are left over by a whole wave: a second launch that splits
    the contraction."""
    m = q()
    wide, deep, gs = 256 * (sms() // 5 + 1), 2048, 64
    rng = np.random.default_rng(M)
    m.q4gsw_debug_pin_routes(gemm=gemm)
    try:
        packed, wg, wu = block(wide // 2, deep, gs, f32s, 45)
        x = rng.standard_normal((M, deep)).astype(np.float16)
        h, gu = m.q4gsw_gated_fwd(packed, wide // 2, deep, gs, cuda(x), act="gelu_tanh", save_gu=True, f32s=f32s)
        assert launches(m.q4gsw_last_route()) == 2 and "rest_splits=" in m.q4gsw_last_route(), m.q4gsw_last_route()
        want_h, want_gu = ol.gated_fwd(x, wg, wu, "gelu_tanh")
        close(h, want_h, "h")
        close(gu, want_gu, "gu")
        only = m.q4gsw_gated_fwd(packed, wide // 2, deep, gs, cuda(x), act="gelu_tanh", f32s=f32s)
        assert torch.equal(only, h)
        packed, wg, wu = block(deep // 2, wide, gs, f32s, 47)
        gu = rng.standard_normal((M, deep)).astype(np.float16)
        d_h = (rng.standard_normal((M, deep // 2)) * 0.05).astype(np.float16)
        d_x, d_gu = m.q4gsw_gated_bwd(packed, deep // 2, wide, gs, cuda(gu), cuda(d_h), f32s=f32s)
        assert launches(m.q4gsw_last_route()) == 3 and "rest_splits=" in m.q4gsw_last_route(), m.q4gsw_last_route()
        want_dx, want_dgu = ol.gated_bwd(gu, d_h, wg, wu, "silu")
        close(d_x, want_dx, "d_x")
        close(d_gu, want_dgu, "d_gu")
    finally:
        m.q4gsw_debug_pin_routes()
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """A seeded draw of sizes, group sizes, scale types, epilogues and kernels, with rows behind the batch."""
    m = q()
    rng = np.random.default_rng(1000 + seed)
    M = int(np.exp(rng.uniform(0, np.log(900))))
    K, gs = 64 * int(rng.integers(1, 17)), int(rng.choice([16, 32, 64]))
    N = 8 * int(np.exp(rng.uniform(0, np.log(200))))
    f32s, kind = bool(rng.integers(2)), str(rng.choice(["none", "silu", "gelu_tanh"]))
    pins = dict(gemv=str(rng.choice(["auto", "tma", "tma_xs"])) if M <= 16 else "auto",
                gemm=str(rng.choice(["auto", "ts", "ss1", "ss2"])) if M > 16 else "auto")
    behind = lambda rows, cols: torch.full((rows + 2, cols), 7.0, dtype=torch.float16, device="cuda")   # noqa: E731
    what = f"M={M} N={N} K={K} gs={gs} f32s={f32s} {kind} {pins}"
    x = rng.standard_normal((M, K)).astype(np.float16)
    bias = rng.standard_normal(N).astype(np.float16) if rng.integers(2) else None
    res = rng.standard_normal((M, N)).astype(np.float16) if rng.integers(2) else None
    d_y = (rng.standard_normal((M, N)) * 0.05).astype(np.float16)
    dev = lambda a: None if a is None else cuda(a)   # noqa: E731
    codes, scales = weight(N, K, gs, f32s, seed)
    w = ol.dequant(codes, scales, gs)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    packed, wg, wu = block(N, K, gs, f32s, 2 * seed)
    m.q4gsw_debug_pin_routes(**pins)
    try:
        y, z, d_x = behind(M, N), behind(M, N), behind(M, K)
        m.q4gsw_linear_act_fwd(blob, N, K, gs, cuda(x), bias=dev(bias), act=kind, residual=dev(res), y=y[:M], z=z[:M],
                               f32s=f32s)
        want_y, want_z = ol.linear_act_fwd(x, w, kind, bias, res)
        close(y[:M], want_y, "y " + what)
        close(z[:M], want_z, "z " + what)
        zz = z[:M] if kind != "none" else None
        _, d_z, d_b = m.q4gsw_linear_act_bwd(blob, N, K, gs, cuda(d_y), z=zz, act=kind, d_x=d_x[:M], want_bias=True,
                                             f32s=f32s)
        want_dx, want_dz, want_db = ol.linear_act_bwd(z[:M].cpu().numpy(), d_y, w, kind)
        close(d_x[:M], want_dx, "d_x " + what)
        close(d_b, want_db, "d_bias " + what)
        if d_z is not None:
            close(d_z, want_dz, "d_z " + what)
        act = "silu" if kind == "none" else kind
        h, gu, d_gu, d_x2 = behind(M, N), behind(M, 2 * N), behind(M, 2 * N), behind(M, K)
        m.q4gsw_gated_fwd(packed, N, K, gs, cuda(x), act=act, h=h[:M], gu=gu[:M], f32s=f32s)
        want_h, want_gu = ol.gated_fwd(x, wg, wu, act)
        close(h[:M], want_h, "h " + what)
        close(gu[:M], want_gu, "gu " + what)
        m.q4gsw_gated_bwd(packed, N, K, gs, gu[:M], cuda(d_y), act=act, d_gu=d_gu[:M], d_x=d_x2[:M], f32s=f32s)
        want_dx, want_dgu = ol.gated_bwd(gu[:M].cpu().numpy(), d_y, wg, wu, act)
        close(d_gu[:M], want_dgu, "d_gu " + what)
        close(d_x2[:M], want_dx, "gated d_x " + what)
        for t in (y, z, d_x, h, gu, d_gu, d_x2):
            assert (t[M:] == 7.0).all(), what
    finally:
        m.q4gsw_debug_pin_routes()
    m.q4gsw_device_error_check()


def test_prepack_gated_refuses_what_is_no_tensor():
    m = q()
    c, s = (cuda(a) for a in weight(64, 128, 32, False, 49))
    with pytest.raises(TypeError, match="packed"):
        m.q4gsw_prepack_gated(c, s, c, s, 32, packed=bytearray(1 << 16))
    with pytest.raises(m.Q4gswError) as e:
        m.q4gsw_prepack_gated(c, s, c, s, 32, packed=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status_name == "Q4GSW_ERR_SIZE"
