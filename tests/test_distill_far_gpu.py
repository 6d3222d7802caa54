"""The distillation operators where a row lies far from zero, against bounds that go by the spread of the row."""
import numpy as np
import pytest
import torch

from helpers import cuda
from oracle import q4gsw_layer as ol
from test_distill_gpu import check, inputs, q

pytestmark = pytest.mark.gpu

OFFSETS = [0.0, 1e3, -2e4, 2e4]


def shifted(M, V, k, offset, seed, **kw):
    """Rows around `offset`, the teacher's too; parts of a row around other values, so that the warps' and the
    CTAs' maxima differ."""
    z, idx, t, d = inputs(M, V, k, seed, half_teacher=False, **kw)
    rng = np.random.default_rng(seed + 1)
    z = z.astype(np.float32) + rng.uniform(-4, 4, (M, V // 8)).astype(np.float32).repeat(8, 1) + np.float32(offset)
    return z, idx, t + np.float32(offset), d


@pytest.mark.parametrize("T", [0.5, 1.0, 1.7])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("M,V,k", [(3, 1024, 8), (5, 32000, 64), (2, 65536, 128), (200, 8192, 16)])
def test_what_a_row_has_in_common_cancels_in_the_one_pass_step(M, V, k, offset, T):
    m = q()
    T = float(np.float32(T))
    z, idx, t, d = shifted(M, V, k, offset, 21, dup=True)
    loss, lse, g = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T)
    assert "launches=1" in m.q4gsw_last_route()
    _, want_lse, want_g = ol.distill_spread(z, idx, t, T, d)
    check(lse, want_lse, "lse")
    check(g, want_g, "d_logits")
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("M,V", [(1, 262144), (800, 49152)])
def test_many_tiles_a_row_far_from_zero(M, V, offset):
    """A CTA of the loss walks several tiles, in which its running maximum grows."""
    m = q()
    T, k = 0.5, 20
    z, idx, t, d = shifted(M, V, k, offset, 22)
    z = np.sort(z.reshape(M, -1, 4096), axis=1).reshape(M, V)      # from tile to tile
    _, lse = m.q4gsw_distill_fwd(cuda(z), cuda(idx), cuda(t), temperature=T)
    assert "tiles=1" not in m.q4gsw_last_route().split()
    rows = slice(0, 4)
    check(lse[rows], ol.distill_spread(z[rows], idx[rows], t[rows], T)[1], "lse")
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("T", [0.5, 1.0, 1.7])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("M,V,k", [(3, 1024, 8), (5, 32000, 64), (1, 262144, 200), (2, 32000, 1024)])
def test_what_a_row_has_in_common_cancels_in_the_loss(M, V, k, offset, T):
    """The loss is a difference of the two distributions; neither side's distance from zero is in it."""
    m = q()
    T = float(np.float32(T))
    z, idx, t, d = shifted(M, V, k, offset, 23)
    z[0] = np.float32(offset) - np.float32(30)
    z[0, idx[0]] = t[0]                        # a student that agrees: a loss near zero
    loss, lse = m.q4gsw_distill_fwd(cuda(z), cuda(idx), cuda(t), temperature=T)
    want_loss, want_lse, _ = ol.distill_spread(z, idx, t, T)
    check(lse, want_lse, "lse")
    check(loss, want_loss, "loss")
    loss, _, _ = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T)
    check(loss, want_loss, "loss of the step")


def test_the_loss_of_a_row_masked_whole_by_the_lowest_value():
    """Uniform over the vocabulary, although the row's log-sum-exp over T may pass the fp32 range."""
    m = q()
    V, k = 1024, 8
    z = np.full((2, V), np.finfo(np.float32).min, np.float32)
    idx = np.arange(2 * k, dtype=np.int32).reshape(2, k)
    t = np.random.default_rng(24).standard_normal((2, k)).astype(np.float32)
    for T in (0.5, 1.0, 2.0):
        e = np.exp(t.astype(np.float64) / T)
        p = e / e.sum(1, keepdims=True)
        want = T * T * (p * (np.log(p) + np.log(V))).sum(1)
        loss, _ = m.q4gsw_distill_fwd(cuda(z), cuda(idx), cuda(t), temperature=T)
        assert np.abs(loss.cpu().numpy() - want).max() <= 2.0 ** -18 * T * T * np.log(V), T


TWO_LAUNCHES = [(3, 1024, 200, True), (5, 32000, 64, True), (2, 65544, 17, False), (3, 8200, 512, False),
                (1, 262144, 20, True), (300, 16392, 8, True)]


@pytest.mark.parametrize("T", [0.5, 1.7])
@pytest.mark.parametrize("offset", [0.0, -2e4, 2e4])
@pytest.mark.parametrize("M,V,k,half", TWO_LAUNCHES)
def test_what_a_row_has_in_common_cancels_in_the_step_of_two_launches(M, V, k, half, offset, T):
    m = q()
    T = float(np.float32(T))
    z, idx, t, d = shifted(M, V, k, offset, 25, dup=True)
    z = z.astype(np.float16 if half else np.float32)
    out = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T)
    assert "launches=2" in m.q4gsw_last_route()
    rows = slice(0, 8)
    want = ol.distill_spread(z[rows], idx[rows], t[rows], T, d[rows], two=True)
    for got, ref, what in zip(out, want, ("loss", "lse", "d_logits")):
        check(got[rows], ref, what)
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("k", [8, 200])
def test_the_step_on_a_row_masked_whole(half, k):
    """All logits at the type's lowest value: uniform probabilities from one launch and from two."""
    m = q()
    V = 1024
    z = np.full((2, V), np.finfo(np.float16 if half else np.float32).min, np.float16 if half else np.float32)
    _, idx, t, _ = inputs(2, V, k, 26)
    d = np.array([1.0, 512.0], np.float32)
    for T in (0.5, 1.0, 2.0):
        loss, _, g = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d), temperature=T)
        _, _, want = ol.distill_spread(np.zeros_like(z), idx, t, T, d)     # (the same probabilities)
        check(g, want, "d_logits")
        assert torch.isfinite(loss).all()


@pytest.mark.parametrize("T", [0.5, 1.0, 1.7])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("M,V,k,half", [(3, 1024, 8, False), (5, 32000, 64, True), (2, 70000, 200, False)])
def test_the_gradient_from_a_saved_log_sum_exp(M, V, k, half, offset, T):
    """Of the log-sum-exp as it was saved, however far from zero it is."""
    m = q()
    T = float(np.float32(T))
    z, idx, t, d = shifted(M, V, k, offset, 27, dup=True)
    z = z.astype(np.float16 if half else np.float32)
    _, lse = m.q4gsw_distill_fwd(cuda(z), cuda(idx), cuda(t), temperature=T)
    g = m.q4gsw_distill_bwd(cuda(z), lse, cuda(idx), cuda(t), cuda(d), temperature=T)
    check(g, ol.distill_spread(z, idx, t, T, d, lse.cpu().numpy())[2], "d_logits")


def test_the_longest_vocabulary():
    """V = 2^31 - 8: the number of a row's tiles and every index within the row stay in 32 bits."""
    m = q()
    V = 2 ** 31 - 8
    free, _ = torch.cuda.mem_get_info()
    if free < 16 * 2 ** 30:
        pytest.skip("needs 16 GB")
    z = torch.zeros((1, V), dtype=torch.float16, device="cuda")
    z[0, V - 2] = z[0, 5] = 8.0
    idx = torch.tensor([[0, V - 1]], dtype=torch.int32, device="cuda")
    t = torch.zeros((1, 2), device="cuda")
    total = V - 2 + 2 * np.exp(8.0)
    lse = torch.tensor([np.log(total)], dtype=torch.float32, device="cuda")
    # d_loss 2^14: a token's gradient is a whole number of fp16 steps but for 3e-6 of it
    d = torch.tensor([2.0 ** 14], device="cuda")
    loss, lse2 = m.q4gsw_distill_fwd(z, idx, t)
    assert abs(lse2.item() - np.log(total)) <= 2.0 ** -18 * np.log(total)
    assert abs(loss.item() - (np.log(0.5) + np.log(total))) <= 2.0 ** -18 * np.log(total)
    for g in (m.q4gsw_distill_bwd(z, lse, idx, t, d), m.q4gsw_distill_step(z, idx, t, d)[2]):
        want = np.float16(2.0 ** 14 / total)
        assert abs(2.0 ** 14 / total / float(want) - 1) < 1e-3
        same = (g[0] == float(want)).sum().item()
        assert same == V - 4
        for i, p in ((0, 1 / total - 0.5), (V - 1, 1 / total - 0.5), (5, np.exp(8) / total), (V - 2, np.exp(8) / total)):
            assert abs(g[0, i].item() - 2.0 ** 14 * p) <= 2.0 ** -10 * 2.0 ** 14 * abs(p), i
        del g
    m.q4gsw_device_error_check()


@pytest.mark.parametrize("half", [False, True])
def test_a_row_with_an_infinite_logit_is_nan_and_stays_alone(half):
    m = q()
    z, idx, t, d = inputs(3, 9000, 8, 28, half_logits=half)
    clean = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d))
    z[1, 4000] = np.inf
    out = m.q4gsw_distill_step(cuda(z), cuda(idx), cuda(t), cuda(d))
    for a, b in zip(out, clean):
        assert torch.isnan(a[1]).all() and torch.equal(a[[0, 2]], b[[0, 2]])
    g = m.q4gsw_distill_bwd(cuda(z), out[1], cuda(idx), cuda(t), cuda(d))
    assert torch.isnan(g[1]).all() and torch.isfinite(g[[0, 2]]).all()
