"""The oracle of the layer operators against exact small cases and against
differences: every gradient formula is the derivative of its forward."""
import numpy as np
import pytest

from oracle import q4gsw_layer as ol

KINDS = ("none", "silu", "gelu_tanh")


@pytest.mark.parametrize("kind", KINDS)
def test_slope_is_the_difference_quotient_of_the_activation(kind):
    z = np.linspace(-9, 9, 721)
    d = 1e-5
    diff = (ol.act(z + d, kind) - ol.act(z - d, kind)) / (2 * d)
    assert np.abs(diff - ol.slope(z, kind)).max() < 1e-9
    assert np.abs(ol.slope(z, kind)).max() <= ol.SLOPE_MAX


def _weights(F, K, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (F, K), dtype=np.uint8)
    scales = rng.uniform(0.05, 0.2, (K // 16, F)).astype(np.float16)
    return ol.dequant(codes, scales, 16)


def test_dequant_is_code_minus_8_times_the_group_scale():
    codes = np.array([[8, 9, 0, 15] * 8, [1] * 32], np.uint8)
    scales = np.array([[0.5, 2.0], [0.25, 4.0]], np.float16)
    w = ol.dequant(codes, scales, 16)
    assert list(w[0, :4]) == [0.0, 0.5, -4.0, 3.5] and list(w[0, 16:20]) == [0.0, 0.25, -2.0, 1.75]
    assert w[1, 0] == -14.0 and w[1, 31] == -28.0


@pytest.mark.parametrize("kind", KINDS[1:])
def test_gated_gradient_is_the_difference_quotient(kind):
    rng = np.random.default_rng(3)
    wg, wu = _weights(8, 32, 1), _weights(8, 32, 2)
    x, c = rng.standard_normal((3, 32)), rng.standard_normal((3, 8))
    (_, _), (gu, _) = ol.gated_fwd(x, wg, wu, kind)
    (d_x, _), _ = ol.gated_bwd(gu, c, wg, wu, kind)
    for _ in range(20):
        v = rng.standard_normal(x.shape)
        d = 1e-5
        f = lambda s: (ol.gated_fwd(x + s * v, wg, wu, kind)[0][0] * c).sum()   # noqa: E731
        assert abs((f(d) - f(-d)) / (2 * d) - (d_x * v).sum()) < 1e-6 * (1 + np.abs(d_x * v).sum())


@pytest.mark.parametrize("kind", KINDS)
def test_linear_gradients_are_difference_quotients(kind):
    rng = np.random.default_rng(4)
    w = _weights(8, 32, 5)
    x, c, bias = rng.standard_normal((3, 32)), rng.standard_normal((3, 8)), rng.standard_normal(8)
    (_, _), (z, _) = ol.linear_act_fwd(x, w, kind, bias)
    (d_x, _), (_, _), (d_b, _) = ol.linear_act_bwd(z, c, w, kind)
    for _ in range(20):
        v, vb = rng.standard_normal(x.shape), rng.standard_normal(8)
        d = 1e-5
        f = lambda s: (ol.linear_act_fwd(x + s * v, w, kind, bias + s * vb)[0][0] * c).sum()   # noqa: E731
        want = (d_x * v).sum() + (d_b * vb).sum()
        assert abs((f(d) - f(-d)) / (2 * d) - want) < 1e-6 * (1 + np.abs(d_x * v).sum())


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_distillation_gradient_is_the_difference_quotient(T):
    rng = np.random.default_rng(6)
    M, V, k = 5, 24, 6
    z, t = rng.standard_normal((M, V)) * 2, rng.standard_normal((M, k)) * 2
    idx = np.stack([rng.permutation(V)[:k] for _ in range(M)]).astype(np.int32)
    idx[1, 3:] = -1
    idx[2, 4] = idx[2, 1]       # the same token twice
    idx[3, :] = -1              # nothing left
    t[1, 3:] = np.nan           # not looked at
    t[4, 2] = -np.inf           # a weight of zero
    c = rng.uniform(0.5, 2, M)
    (loss, _), _, (g, _) = ol.distill(z, idx, t, T, c)
    assert loss[3] == 0 and (g[3] == 0).all() and np.isfinite(loss).all()
    assert np.abs(g.sum(1)).max() < 1e-12        # p and q both sum to one
    for _ in range(20):
        v, d = rng.standard_normal(z.shape), 1e-5
        f = lambda s: (ol.distill(z + s * v, idx, t, T)[0][0] * c).sum()   # noqa: E731
        assert abs((f(d) - f(-d)) / (2 * d) - (g * v).sum()) < 1e-6


def test_distillation_loss_is_zero_for_a_student_that_agrees():
    t = np.array([[1.0, 2.0, 0.5]])
    z = np.full((1, 16), -np.inf)
    z[0, [3, 9, 12]] = t[0] + 5.0
    (loss, _), (lse, _), (g, _) = ol.distill(z, np.array([[3, 9, 12]]), t, 2.0, np.ones(1))
    assert abs(loss[0]) < 1e-12 and np.abs(g).max() < 1e-12
    assert abs(lse[0] - np.log(np.exp((t[0] + 5.0) / 2).sum())) < 1e-12


def test_spread_bounds_do_not_grow_with_what_a_row_has_in_common():
    rng = np.random.default_rng(7)
    z, t = rng.integers(-9, 10, (4, 256)) / 4, rng.integers(-9, 10, (4, 12)) / 4      # exact after a shift, too
    idx = np.stack([rng.permutation(256)[:12] for _ in range(4)]).astype(np.int32)
    idx[1, 5:], idx[2, :] = -1, -1
    c = rng.uniform(0.5, 2, 4)
    near, far = (ol.distill_spread(z + s, idx, t + s, 0.5, c) for s in (0.0, 2.0 ** 14))
    for a, b, what in zip(near, far, ("loss", "lse", "d_logits")):
        if what != "lse":
            assert np.abs(a[0] - b[0]).max() < 1e-9
            assert np.abs(a[1] / b[1] - 1).max() < 1e-6, what
