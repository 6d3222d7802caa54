"""The norms around a block on the GPU against the fp64 oracle, forward and
backward, within bounds counted from the kernels' roundings."""
import itertools

import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_adapters as oa

pytestmark = pytest.mark.gpu

FIELDS = ("residual", "block", "gate", "w_post", "w_pre")


def q():
    import bit_group_quantized_q4gsw_b200 as m
    return m


def close(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().numpy().astype(np.float64)
    assert got.shape == value.shape, (what, got.shape, value.shape)
    over = ~(np.abs(got - value) <= bound)
    # fp16's largest value is 65504 and its step there 32: from 65520 on the rounding to nearest is infinite
    over &= ~(np.isinf(got) & (np.sign(got) == np.sign(value)) & (np.abs(value) + bound >= 65520))
    if over.any():
        i = np.unravel_index(np.argmax(np.where(over, np.abs(got - value) / bound, 0)), got.shape)
        raise AssertionError(f"{what}: {over.sum()} of {over.size} outside; worst at {i}: got {got[i]!r} want {value[i]!r} "
                             f"bound {bound[i]!r} [{q().q4gsw_last_route()}]")


def make(M, D, block=True, post=True, gate="feature", pre=True, offset=1.0, f=0.75, eps=1e-6, seed=0):
    g = np.random.default_rng(seed + 7 * M + D)
    n = lambda *s, k=1.0: (g.standard_normal(s) * k).astype(np.float16)      # noqa: E731
    return dict(h=n(M, D, k=3), block=n(M, D, k=0.5) if block else None, w_post=n(D, k=0.3) if block and post else None,
                gate={"none": None, "feature": n(D, k=0.5), "token": n(M, D, k=0.5)}[gate if block else "none"],
                residual_scale=f, w_pre=n(D, k=0.3) if pre else None, eps=eps, weight_offset=offset,
                d_x=n(M, D, k=0.05) if pre else None, d_h=n(M, D, k=0.05))


def on_gpu(c):
    return {k: cuda(v) if isinstance(v, np.ndarray) else v for k, v in c.items() if k not in ("h", "d_x", "d_h")}


def check(c, weights=True):
    m = q()
    how = on_gpu(c)
    plain = {k: v for k, v in c.items() if k not in ("d_x", "d_h")}
    x, s = m.q4gsw_norms_fwd(cuda(c["h"]), **how)
    want_x, want_s = oa.norms_fwd(**plain)
    close(s, want_s, "h'")
    if want_x is None:
        assert x is None
    else:
        close(x, want_x, "x")
    d_x = None if c["d_x"] is None else cuda(c["d_x"])
    d_h = None if c["d_h"] is None else cuda(c["d_h"])
    got = m.q4gsw_norms_bwd(s, d_x=d_x, d_h=d_h, want_weights=weights, **how)
    want = oa.norms_bwd(s.cpu().numpy(), c["d_x"], c["d_h"], **{k: v for k, v in plain.items() if k != "h"})
    sums = {"w_post", "w_pre"} | ({"gate"} if c["gate"] is not None and c["gate"].ndim == 1 else set())
    for k in FIELDS:
        v = getattr(got, k)
        if k in want and (weights or k not in sums):
            close(v, want[k], k)
        else:
            assert v is None, k
    return x, s, got


# every width rule, odd widths among them; few and many rows
@pytest.mark.parametrize("D", [8, 64, 256, 264, 1000, 1024, 2048, 2056, 4096, 4104, 8192, 8200, 14336, 16384, 16392, 32768])
@pytest.mark.parametrize("M", [1, 3, 37])
def test_widths(M, D):
    check(make(M, D))
    check(make(M, D, gate="token"), weights=False)


@pytest.mark.parametrize("M,D", [(512, 2048), (1021, 512), (700, 72), (2000, 4096), (300, 16384)])
def test_many_rows(M, D):
    check(make(M, D))
    check(make(M, D, gate="none"), weights=False)


@pytest.mark.parametrize("block,post,gate,pre", [p for p in itertools.product(
    (False, True), (False, True), ("none", "feature", "token"), (False, True)) if p[0] or (not p[1] and p[2] == "none")])
@pytest.mark.parametrize("weights", [False, True])
def test_every_form(block, post, gate, pre, weights):
    for offset, f in ((0.0, 1.0), (1.0, -0.5)):
        if not block and not pre and f == 1.0:
            continue
        check(make(19, 328, block, post, gate, pre, offset, f), weights)


def test_gradients_from_one_side_alone():
    c = make(9, 200)
    c["d_h"] = None
    check(c)
    c = make(9, 200, pre=False)
    check(c)


def test_rows_of_zeros_and_extreme_rows():
    c = make(6, 512, gate="none", eps=1e-6)
    c["block"][0] = 0                       # a row whose mean square is 0
    c["h"][1], c["block"][1] = 0, 0
    c["block"][2], c["h"][2] = 60000, -60000
    c["block"][3] = np.float16(6e-8)        # the least fp16 value: far below eps
    c["h"][4] = 6e-8
    check(c)
    c["eps"] = 1e-2
    check(c)


@pytest.mark.parametrize("D", [512, 16384])
def test_rows_of_zeros_and_an_eps_whose_factor_leaves_fp32_in_its_cube(D):
    c = make(4, D, eps=1e-30)               # rsqrt(eps)^3 = 1e45
    c["h"][1], c["block"][1] = 0, 0         # both norms' rows
    c["block"][2] = 0
    check(c)


def test_a_row_that_is_not_finite_stays_alone():
    m = q()
    c = make(8, 264)
    how = on_gpu(c)
    h = cuda(c["h"])
    x, s = m.q4gsw_norms_fwd(h, **how)
    d = m.q4gsw_norms_bwd(s, d_x=cuda(c["d_x"]), d_h=cuda(c["d_h"]), **how)
    how["block"][3, 5], h[6, 0], how["block"][1, 7] = float("nan"), float("inf"), float("-inf")
    x2, s2 = m.q4gsw_norms_fwd(h, **how)
    rest = [0, 2, 4, 5, 7]
    assert torch.equal(x2[rest], x[rest]) and torch.equal(s2[rest], s[rest])
    assert torch.isnan(x2[3]).all() and torch.isnan(x2[1]).any() and torch.isinf(s2[6, 0])
    d2 = m.q4gsw_norms_bwd(s2, d_x=cuda(c["d_x"]), d_h=cuda(c["d_h"]), **how)
    assert torch.equal(d2.residual[rest], d.residual[rest]) and torch.equal(d2.block[rest], d.block[rest])


def test_in_place():
    m = q()
    c = make(33, 520, gate="token")
    how = on_gpu(c)
    h = cuda(c["h"])
    x, s = m.q4gsw_norms_fwd(h, **how)
    x2, s2 = m.q4gsw_norms_fwd(h, h_out=h, **how)
    assert s2 is h and torch.equal(h, s) and torch.equal(x, x2)
    d_x, d_h = cuda(c["d_x"]), cuda(c["d_h"])
    d = m.q4gsw_norms_bwd(s, d_x=d_x, d_h=d_h, want_weights=True, **how)
    both = d_h.clone()
    block, gate = how.pop("block"), how.pop("gate")
    e = m.q4gsw_norms_bwd(s, d_x=d_x, d_h=both, block=block, gate=gate, d_block=block, d_gate=gate, d_residual=both,
                          want_weights=True, **how)
    assert e.residual is both and e.block is block and e.gate is gate
    assert all(torch.equal(getattr(d, k), getattr(e, k)) for k in FIELDS)


def test_the_pre_norm_alone_returns_the_stream_itself():
    m = q()
    c = make(5, 128, block=False, f=1.0)
    h = cuda(c["h"])
    x, s = m.q4gsw_norms_fwd(h, w_pre=cuda(c["w_pre"]), weight_offset=1.0)
    assert s is h
    buf = torch.empty_like(h)
    x2, s2 = m.q4gsw_norms_fwd(h, w_pre=cuda(c["w_pre"]), weight_offset=1.0, h_out=buf)
    assert s2 is buf and torch.equal(buf, h) and torch.equal(x, x2)
    with pytest.raises(ValueError, match="nothing to compute"):
        m.q4gsw_norms_fwd(h)


def test_empty_batch():
    m = q()
    w = torch.ones(64, device="cuda").half()
    e = torch.empty(0, 64, device="cuda").half()
    x, s = m.q4gsw_norms_fwd(e, block=e, w_post=w, gate=w, w_pre=w)
    assert x.shape == s.shape == (0, 64)
    d = m.q4gsw_norms_bwd(s, d_x=e, d_h=e, block=e, w_post=w, gate=w, w_pre=w, want_weights=True)
    assert d.residual.shape == (0, 64) and not d.w_pre.any() and not d.w_post.any() and not d.gate.any()


def test_repeats_streams_and_graphs():
    m = q()
    c = make(700, 1032)
    how = on_gpu(c)
    h, d_x, d_h = cuda(c["h"]), cuda(c["d_x"]), cuda(c["d_h"])

    def both():
        x, s = m.q4gsw_norms_fwd(h, **how)
        return (x, s, *m.q4gsw_norms_bwd(s, d_x=d_x, d_h=d_h, want_weights=True, **how))

    want = both()
    for _ in range(20):
        assert all(torch.equal(v, w) for v, w in zip(both(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(v, w) for v, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    h.copy_(torch.randn_like(h))
    graph.replay()
    assert all(torch.equal(v, w) for v, w in zip(got, both()))


def test_offsets_past_2_31_elements():
    m = q()
    M, D = 65600, 32768
    h = torch.empty(M, D, device="cuda", dtype=torch.float16).normal_()
    w = torch.randn(D, device="cuda").half()
    x, s = m.q4gsw_norms_fwd(h, block=h, w_post=w, w_pre=w)
    rows = [0, 1, 32768, 65535, 65536, M - 1]
    some = h[rows].cpu().numpy()
    want_x, want_s = oa.norms_fwd(some, block=some, w_post=w.cpu().numpy(), w_pre=w.cpu().numpy())
    close(x[rows], want_x, "x")
    close(s[rows], want_s, "h'")
    del x
    d = m.q4gsw_norms_bwd(s, d_x=h, block=h, w_post=w, w_pre=w)
    want = oa.norms_bwd(s[rows].cpu().numpy(), some, None, some, w.cpu().numpy(), w_pre=w.cpu().numpy())
    close(d.residual[rows], want["residual"], "residual")
    close(d.block[rows], want["block"], "block")


def test_python_checks():
    m = q()
    h, w = torch.zeros(4, 64, device="cuda").half(), torch.zeros(64, device="cuda").half()
    for kw, what in ((dict(w_post=w), "without a block"), (dict(gate=w), "without a block"), (dict(block=h[:2], w_pre=w), "block must"),
                     (dict(block=h, gate=torch.zeros(2, 64, device="cuda").half()), "gate must"), (dict(block=h, x=h), "x needs")):
        with pytest.raises(ValueError, match=what):
            m.q4gsw_norms_fwd(h, **kw)
    for kw, what in ((dict(d_x=h), "go together"), (dict(d_h=h, w_pre=w), "go together"), (dict(), "d_x or d_h"),
                     (dict(d_h=h, d_block=h), "d_block"), (dict(d_x=h, w_pre=w, d_gate=w), "d_gate"), (dict(d_h=h, d_w_post=w), "d_w_post")):
        with pytest.raises(ValueError, match=what):
            m.q4gsw_norms_bwd(h, **kw)
    with pytest.raises(m.Q4gswError, match="SHAPE"):
        m.q4gsw_norms_fwd(h, w_pre=w, eps=-1.0)
