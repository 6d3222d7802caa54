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
