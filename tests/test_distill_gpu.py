"""The distillation loss, log-sum-exp and gradient against the fp64 oracle."""
import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_layer as ol

pytestmark = pytest.mark.gpu


def q():
    import bit_group_quantized_q4gsw_b200 as m
    return m


def inputs(M, V, k, seed, half_logits=False, half_teacher=True, pad=False, dup=False):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((M, V)) * 3).astype(np.float16 if half_logits else np.float32)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(M)]).astype(np.int32)
    t = (rng.standard_normal((M, k)) * 2 + 8).astype(np.float16 if half_teacher else np.float32)
    if pad:
        n = rng.integers(0, k + 1, M)
        n[0] = 0
        for r in range(M):
            idx[r, n[r]:] = -1
            t[r, n[r]:] = [np.nan, np.inf, -np.inf][r % 3]
    if dup and k > 1:
        idx[:, k // 2] = idx[:, 0]
    d = rng.uniform(0.5, 1.5, M).astype(np.float32) * 4
    return z, idx, t, d


def check(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().numpy().astype(np.float64)
    over = ~(np.abs(got - value) <= bound)
    if over.any():
        i = np.unravel_index(np.argmax(np.abs(got - value) / bound), got.shape)
        raise AssertionError(f"{what}: {over.sum()} outside; worst at {i}: got {got[i]!r} want {value[i]!r} "
                             f"bound {bound[i]!r} [{q().q4gsw_last_route()}]")


# vocabularies of one vector, below, at and past one CTA's tile, past a cluster
# of eight (streamed); one row and many; a list longer than a CTA has threads
CASES = [
    (1, 8, 1, 1.0, False, False), (3, 8, 8, 2.0, True, True), (5, 264, 20, 0.5, False, True),
    (1, 2048, 1, 1.0, False, True), (2, 8192, 64, 2.0, False, True), (3, 8200, 64, 1.0, True, False),
    (7, 32000, 100, 1.5, False, True), (40, 32000, 64, 2.0, True, True), (1, 32000, 512, 3.0, False, False),
    (2, 65536, 17, 1.0, False, True), (2, 65544, 33, 1.0, False, True), (1, 131080, 1024, 2.0, True, False),
    (3, 262144, 20, 1.0, False, False), (700, 1024, 10, 4.0, False, True),
]


@pytest.mark.parametrize("M,V,k,T,half_logits,half_teacher", CASES)
def test_loss_and_gradient(M, V, k, T, half_logits, half_teacher):
    m = q()
    for pad, dup in ((False, False), (True, False), (False, True)):
        z, idx, t, d = inputs(M, V, k, M + V + k, half_logits, half_teacher, pad, dup)
        dz, di, dt, dd = cuda(z), cuda(idx), cuda(t), cuda(d)
        loss, lse = m.q4gsw_distill_fwd(dz, di, dt, temperature=T)
        want_loss, want_lse, want_g = ol.distill(z, idx, t, T, d)
        check(lse, want_lse, "lse")
        check(loss, want_loss, "loss")
        loss2, lse2, g = m.q4gsw_distill_step(dz, di, dt, dd, temperature=T)
        # (another split of the row, so another order of the same sums)
        check(lse2, want_lse, "lse of the step")
        check(loss2, want_loss, "loss of the step")
        check(g, want_g, "d_logits of the step")
        g2 = m.q4gsw_distill_bwd(dz, lse, di, dt, dd, temperature=T)
        check(g2, ol.distill(z, idx, t, T, d, lse.cpu().numpy())[2], "d_logits of the backward")
        if pad:
            assert loss[0] == 0 and (g[0] == 0).all() and (g2[0] == 0).all()
    m.q4gsw_device_error_check()


def test_masked_and_extreme_logits():
    m = q()
    M, V, k = 6, 1000, 8
    z, idx, t, d = inputs(M, V, k, 5)
    z[0, :500] = -np.inf                       # half of the vocabulary masked
    z[1, :] = -np.inf
    z[1, idx[1, 0]] = 3.0                      # one token left
    idx[1, 1:] = -1
    z[2] = np.finfo(np.float32).min            # all at the lowest value: uniform
    z[3, :] += 1e4                             # large logits, small differences
    z[4, :] = np.finfo(np.float32).min         # masked by the lowest value but for ten tokens
    z[4, idx[4]] = np.arange(k)
    t[5, 3] = -np.inf                          # a teacher weight of zero on a masked token
    z[5, idx[5, 3]] = -np.inf
    keep = (z[0, idx[0]] == -np.inf)
    idx[0, keep] = -1
    loss, lse, g = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=1.0)
    want_loss, want_lse, want_g = ol.distill(z, idx, t, 1.0, d)
    assert torch.isfinite(loss[[0, 1, 3, 4, 5]]).all()
    rows = [0, 1, 3, 4, 5]
    check(loss[rows], (want_loss[0][rows], want_loss[1][rows]), "loss")
    check(lse[rows], (want_lse[0][rows], want_lse[1][rows]), "lse")
    check(g[rows], (want_g[0][rows], want_g[1][rows]), "d_logits")
    p = g[2].float().cpu().numpy() / d[2]      # uniform probabilities but for the teacher's tokens
    others = np.setdiff1d(np.arange(V), idx[2])
    assert np.abs(p[others] - 1e-3).max() < 1e-6
    # a row of nothing but -infinity, and one with a NaN, are NaN; the others are not touched by them
    z[0, :] = -np.inf
    z[3, 7] = np.nan
    loss2, lse2, g2 = m.q4gsw_distill_step(cuda(z), cuda(np.abs(idx)), cuda(np.nan_to_num(t, neginf=0)), cuda(d))
    assert torch.isnan(loss2[[0, 3]]).all() and torch.isnan(lse2[[0, 3]]).all() and torch.isnan(g2[3]).all()
    assert torch.isfinite(lse2[[1, 4, 5]]).all()


def test_a_teacher_weight_on_a_masked_token_gives_an_infinite_loss_and_a_finite_gradient():
    m = q()
    z = torch.zeros(1, 64, device="cuda")
    z[0, 5] = float("-inf")
    idx = torch.tensor([[5, 6]], dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 2, device="cuda")
    loss, lse, g = m.q4gsw_distill_step(z, idx, t, torch.ones(1, device="cuda"))
    assert loss[0] == float("inf") and torch.isfinite(lse).all() and torch.isfinite(g).all()
    assert abs(g[0, 5].item() + 0.5) < 1e-3 and abs(g[0, 6].item() - (1 / 63 - 0.5)) < 1e-3


@pytest.mark.parametrize("T", [0.5, 2.0])
@pytest.mark.parametrize("offset", [0.0, -2e4, 2e4])
def test_parts_of_a_row_masked_whole(T, offset):
    """The gradient of one pass is a factor away from weights against a part's own maximum: parts that are masked
    whole, with -infinity or with the type's lowest value, beside parts far from zero."""
    m = q()
    V, k = 32000, 16
    rng = np.random.default_rng(int(abs(offset)) + int(4 * T))
    base = (rng.standard_normal((4, V)) * 3 + offset).astype(np.float32)
    masks = [(0, 0), (0, 8000), (0, 24000), (8000, 16000)]
    idx = (24000 + np.stack([rng.permutation(8000)[:k] for _ in masks])).astype(np.int32)
    t = (rng.standard_normal((4, k)) * 2).astype(np.float32)
    d = rng.uniform(0.5, 1.5, 4).astype(np.float32)
    out = []
    for fill in (-np.inf, np.finfo(np.float32).min):
        z = base.copy()
        for r, (lo, hi) in enumerate(masks):
            z[r, lo:hi] = fill
        out.append(m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T))
        assert "launches=1" in m.q4gsw_last_route()
        if fill == -np.inf:
            for got, want, what in zip(out[0], ol.distill(z, idx, t, T, d), ("loss", "lse", "d_logits")):
                check(got, want, what)
    for a, b in zip(*out):      # a masked token weighs nothing either way
        assert torch.equal(a, b)
    for r, (lo, hi) in enumerate(masks):
        assert (out[0][2][r, lo:hi] == 0).all()
    m.q4gsw_device_error_check()


def test_ids_out_of_range_count_as_padding_and_are_reported():
    m = q()
    M, V, k = 4, 256, 6
    z, idx, t, d = inputs(M, V, k, 9)
    want = ol.distill(z, np.where(np.arange(k) == 2, -1, idx), t, 1.0, d)
    for bad in (V, -2, 2 ** 31 - 1, -2 ** 31):
        wrong = idx.copy()
        wrong[:, 2] = bad
        m.q4gsw_device_error_check()
        loss, lse, g = m.q4gsw_distill_step(cuda(z), cuda(wrong), cuda(t), cuda(d))
        with pytest.raises(m.Q4gswError) as e:
            m.q4gsw_device_error_check()
        assert e.value.status_name == "Q4GSW_ERR_INDEX"
        m.q4gsw_device_error_check()
        check(loss, want[0], "loss")
        check(g, want[2], "d_logits")


def test_gradient_against_differences_of_the_loss():
    m = q()
    M, V, k, T = 4, 512, 12, 2.0
    z, idx, t, d = inputs(M, V, k, 11, pad=True)
    _, _, g = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T)
    g = g.cpu().numpy().astype(np.float64)
    bound = ol.distill(z, idx, t, T, d)[2][1]
    rng = np.random.default_rng(12)
    z = z.astype(np.float64)
    for _ in range(5):
        v, s = rng.standard_normal(z.shape), 1e-4
        f = lambda a: (ol.distill(z + a * v, idx, t, T)[0][0] * d).sum()   # noqa: E731
        assert abs((f(s) - f(-s)) / (2 * s) - (g * v).sum()) <= (bound * np.abs(v)).sum() + 1e-6


def test_rows_behind_the_batch_are_left_alone():
    m = q()
    for M, V in ((1, 8), (3, 32000), (2, 70000)):
        z, idx, t, d = inputs(M, V, 4, 13)
        g = torch.full((M + 1, V), 7.0, dtype=torch.float16, device="cuda")
        loss = torch.full((M + 1,), 7.0, device="cuda")
        lse = torch.full((M + 1,), 7.0, device="cuda")
        m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), loss=loss[:M], lse=lse[:M], d_logits=g[:M])
        m.q4gsw_distill_bwd(cuda(z), lse[:M], cuda(idx), cuda(t), cuda(d), d_logits=g[:M])
        assert (g[M] == 7).all() and loss[M] == 7 and lse[M] == 7 and (g[:M] != 7).all()


def test_an_empty_batch():
    m = q()
    e = torch.empty((0, 64), device="cuda")
    i, t = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, lse, g = m.q4gsw_distill_step(e, i, t, torch.empty(0, device="cuda"))
    assert loss.shape == lse.shape == (0,) and g.shape == (0, 64)


@pytest.mark.parametrize("M,V,half", [(300, 32000, False), (2, 262144, False), (64, 65536, True)])
def test_repeats_streams_and_graphs_give_the_same_bits(M, V, half):
    m = q()
    z, idx, t, d = inputs(M, V, 32, 14, half_logits=half, dup=True)
    z, idx, t, d = cuda(z), cuda(idx), cuda(t), cuda(d)
    step = lambda: m.q4gsw_distill_step(z, idx, t, d, temperature=2.0)   # noqa: E731
    first = step()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(step(), first))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([step() for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for r in o for a, b in zip(r, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    z.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    m.q4gsw_device_error_check()


def test_offsets_beyond_32_bits():
    """A batch whose logits pass 2^31 elements: the last rows are read and written at their own places."""
    m = q()
    V, k = 262144, 4
    M = 2 ** 31 // V + 2
    z = torch.zeros((M, V), dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(15)
    tail = (rng.standard_normal((2, V)) * 3).astype(np.float16)
    z[-2:] = cuda(tail)
    idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(M, 1).contiguous()
    t = torch.zeros((M, k), device="cuda")
    d = torch.full((M,), 100.0, device="cuda")
    loss, lse, g = m.q4gsw_distill_step(z, idx, t, d)
    want = ol.distill(tail, idx[-2:].cpu().numpy(), np.zeros((2, k)), 1.0, np.full(2, 100.0))
    check(loss[-2:], want[0], "loss")
    check(g[-2:], want[2], "d_logits")
    g2 = m.q4gsw_distill_bwd(z, lse, idx, t, d)
    check(g2[-2:], ol.distill(tail, idx[-2:].cpu().numpy(), np.zeros((2, k)), 1.0, np.full(2, 100.0),
                              lse[-2:].cpu().numpy())[2], "d_logits of the backward")


def test_a_training_step_from_logits_to_the_input_gradient():
    """Head logits from the packed weight, the distillation gradient, and the head's input gradient."""
    m = q()
    M, V, K, gs, k, T = 48, 1000, 256, 32, 16, 2.0
    rng = np.random.default_rng(16)
    codes = rng.integers(0, 16, (V, K), dtype=np.uint8)
    scales = rng.uniform(0.005, 0.02, (K // gs, V)).astype(np.float16)
    w = ol.dequant(codes, scales, gs)
    x = rng.standard_normal((M, K)).astype(np.float16)
    _, idx, t, d = inputs(M, V, k, 17, pad=True)
    blob = m.q4gsw_prepack(cuda(codes), cuda(scales), gs)
    z = m.q4gsw_linear_fwd(blob, V, K, gs, cuda(x))
    loss, lse, g = m.q4gsw_distill_step(z, cuda(idx), cuda(t), cuda(d), temperature=T)
    d_x = m.q4gsw_linear_bwd_input(blob, V, K, gs, g)
    want_loss, _, want_g = ol.distill(z.cpu().numpy(), idx, t, T, d)
    check(loss, want_loss, "loss")
    check(g, want_g, "d_logits")
    ref = g.cpu().numpy().astype(np.float64) @ w
    assert (np.abs(d_x.cpu().numpy() - ref) <= 4e-3 * (np.abs(g.cpu().numpy().astype(np.float64)) @ np.abs(w)) + 1e-12).all()
    m.q4gsw_device_error_check()
