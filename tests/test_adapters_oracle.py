"""The oracle of the adapters, the norms and the clip against differences and
exact small cases: every gradient is the derivative of its forward."""
import numpy as np
import pytest

from oracle import q4gsw_adapters as oa


def _case(seed=0, M=7, K=12, N=10, L=3, r=4):
    g = np.random.default_rng(seed)
    ids = np.array([1, -1, 0, 1, 1, -1, 0])[:M]          # adapter 2 has no token
    n = g.standard_normal
    return dict(x=n((M, K)), w=n((N, K)), ids=ids, a=n((L, r, K)), b=n((L, N, r)), scale=g.uniform(0.5, 2, L)), n((M, N))


def test_adapters_forward_token_by_token():
    c, _ = _case()
    bias, res = np.arange(10.0), np.ones((7, 10))
    (y, _), (u, _) = oa.adapters_fwd(**c, bias=bias, residual=res)
    for m, i in enumerate(c["ids"]):
        want = c["w"] @ c["x"][m] + bias + res[m]
        if i >= 0:
            assert np.allclose(u[m], c["a"][i] @ c["x"][m])
            want = want + c["scale"][i] * (c["b"][i] @ (c["a"][i] @ c["x"][m]))
        else:
            assert not u[m].any()
        assert np.allclose(y[m], want)


def test_adapters_gradients_are_difference_quotients():
    c, d_y = _case()
    f = lambda **k: (oa.adapters_fwd(**{**c, **k})[0][0] * d_y).sum()   # noqa: E731
    u = oa.adapters_fwd(**c)[1][0]
    (d_x, _), (d_a, _), (d_b, _) = oa.adapters_bwd(c["x"], u, d_y, c["w"], c["ids"], c["a"], c["b"], c["scale"])
    g = np.random.default_rng(1)
    for name, d in (("x", d_x), ("a", d_a), ("b", d_b)):
        for _ in range(8):
            v, h = g.standard_normal(d.shape), 1e-5
            diff = (f(**{name: c[name] + h * v}) - f(**{name: c[name] - h * v})) / (2 * h)
            assert abs(diff - (d * v).sum()) < 1e-6 * (1 + np.abs(d * v).sum()), name
    assert not d_a[2].any() and not d_b[2].any()


def test_a_planted_mistake_fails_the_difference():
    c, d_y = _case()
    u = oa.adapters_fwd(**c)[1][0]
    right = oa.adapters_bwd(c["x"], u, d_y, c["w"], c["ids"], c["a"], c["b"], c["scale"])
    wrong = oa.adapters_bwd(c["x"], u, d_y, c["w"], c["ids"], c["a"], c["b"], None)      # the factor left out
    for (p, b), (v, _) in zip(right, wrong):
        assert (np.abs(p - v) > b).any()


def test_plan_is_a_stable_sort():
    order, first = oa.plan([2, -1, 0, 2, 9, 0], 3)
    assert order == [2, 5, 0, 3, 1, 4] and first == [0, 2, 2, 4, 6]


@pytest.mark.parametrize("gate", ["none", "feature", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norms_gradients_are_difference_quotients(gate, post, offset):
    g = np.random.default_rng(5)
    M, D = 3, 16
    n = g.standard_normal
    c = dict(h=n((M, D)), block=n((M, D)), w_post=n(D) if post else None, w_pre=n(D), residual_scale=0.7, eps=1e-3,
             weight_offset=offset, gate={"none": None, "feature": n(D), "token": n((M, D))}[gate])
    d_x, d_h = n((M, D)), n((M, D))

    def f(**k):
        (x, _), (s, _) = oa.norms_fwd(**{**c, **k})
        return (x * d_x).sum() + (s * d_h).sum()

    s = oa.norms_fwd(**c)[1][0]
    got = oa.norms_bwd(s, d_x, d_h, **{k: v for k, v in c.items() if k != "h"})
    names = dict(residual="h", block="block", gate="gate", w_post="w_post", w_pre="w_pre")
    assert set(got) == {k for k, v in names.items() if c[v] is not None}
    for k, (d, _) in got.items():
        name = names[k]
        for _ in range(6):
            v, h = n(c[name].shape), 1e-5
            diff = (f(**{name: c[name] + h * v}) - f(**{name: c[name] - h * v})) / (2 * h)
            assert abs(diff - (d * v).sum()) < 1e-6 * (1 + np.abs(d * v).sum()), k


def test_norm_of_a_constant_row_by_hand():
    (x, _), (s, _) = oa.norms_fwd(np.full((1, 8), 3.0), block=np.full((1, 8), -2.0), w_post=np.ones(8), residual_scale=2.0,
                                  w_pre=np.full(8, 0.5), eps=0.0)
    assert np.allclose(s, 5.0) and np.allclose(x, 0.5)          # 2 * 3 + (-2 / 2), and 5 / 5 * 0.5


def test_clip_by_hand():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    assert oa.grad_norm(g, 0.5)[0] == 2.5
    outs = oa.grad_clip(g, 1.25, 0.5)
    k = 0.5 * 1.25 / (2.5 + 1e-6)
    assert np.allclose(outs[0][0], [3 * k, 0]) and np.allclose(outs[1][0], [[4 * k]])
    assert np.allclose(oa.grad_clip(g, 9.0)[1][0], [[4.0]])
