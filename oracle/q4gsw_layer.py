"""Plain CPU oracle for the operators around the q4gsw linear layer: the gated
feed-forward block, the projection with an epilogue and the distillation loss.

TEST INFRASTRUCTURE ONLY, under the same rule as ``q4gsw_oracle``.  Everything
is computed in fp64 from the definitions.  Each function returns (value,
bound) pairs; a bound is how far a kernel may be from the value, counted from
the roundings its arithmetic makes:

  EPS_W  2^-11 + 2^-13: the tensor-core operand fp16((code - 8) scale) is off
         by at most half a step, 2^-11 of itself (the GEMV forward rounds no
         weight); fp32 accumulation over a contraction of C terms adds at most
         C 2^-24 of the absolute products, 2^-13 for C <= 2048 (larger C: as
         counted in ``eps_of``);
  HALF   2^-11 relative: one rounding to fp16, and 2^-25 absolute, half the
         smallest fp16 step;
  ACT    2^-18: the fast exponential is within 2^-20 of its value for the
         arguments that matter (2 + 1.2 |x| units of 2^-24), the quotient
         within 2^-22, and at most six fp32 operations follow on terms no
         larger than 1.2.
"""
from __future__ import annotations

import math

import numpy as np

HALF = 2.0 ** -11
TINY = 2.0 ** -25
ACT = 2.0 ** -18
SLOPE_MAX = 1.13   # of silu (1.0998) and gelu_tanh (1.1290)


def eps_of(contraction: int) -> float:
    return 2.0 ** -11 + max(contraction, 2048) * 2.0 ** -24


def dequant(codes, scales, gs):
    """(code - 8) * scale in fp64; scales [K/gs, N] of any float type."""
    s = np.repeat(np.asarray(scales, np.float64), gs, axis=0).T
    return (np.asarray(codes, np.float64) - 8.0) * s


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))


def slope(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return np.ones_like(z)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _rounded(v, err):
    """Bound of an fp16 output of value v whose fp32 value is off by at most err."""
    return err + HALF * (np.abs(v) + err) + TINY


def gated_fwd(x, wg, wu, kind):
    """((h, bound), (gu, bound)); wg, wu [F, K] dequantised."""
    x = np.asarray(x, np.float64)
    e = eps_of(x.shape[1])
    g, u = x @ wg.T, x @ wu.T
    dg, du = e * (np.abs(x) @ np.abs(wg).T), e * (np.abs(x) @ np.abs(wu).T)
    a = act(g, kind)
    h = a * u
    err = SLOPE_MAX * dg * (np.abs(u) + du) + (np.abs(a) * (1 + ACT) + TINY) * du + ACT * np.abs(h) + TINY * np.abs(u)
    gu = np.stack([g, u], 2).reshape(x.shape[0], -1)
    return (h, _rounded(h, err)), (gu, _rounded(gu, np.stack([dg, du], 2).reshape(gu.shape)))


def gated_bwd(gu, d_h, wg, wu, kind):
    """((d_x, bound), (d_gu, bound))."""
    gu, d_h = np.asarray(gu, np.float64), np.asarray(d_h, np.float64)
    g, u = gu[:, 0::2], gu[:, 1::2]
    d_g, d_u = d_h * u * slope(g, kind), d_h * act(g, kind)
    e_g = ACT * np.abs(d_h * u) + 2.0 ** -22 * np.abs(d_g)
    e_u = ACT * np.abs(d_u) + TINY * np.abs(d_h)
    d_gu = np.stack([d_g, d_u], 2).reshape(gu.shape)
    b_gu = _rounded(d_gu, np.stack([e_g, e_u], 2).reshape(gu.shape))
    w = np.stack([wg, wu], 1).reshape(gu.shape[1], -1)
    return _product(d_gu, b_gu, w), (d_gu, b_gu)


def _product(a, b_a, w):
    """(a @ w, bound) for a known to within b_a, fp16 output."""
    e = eps_of(w.shape[0])
    v = a @ w
    return v, _rounded(v, e * ((np.abs(a) + b_a) @ np.abs(w)) + b_a @ np.abs(w))


def linear_act_fwd(x, w, kind, bias=None, residual=None):
    """((y, bound), (z, bound))."""
    x = np.asarray(x, np.float64)
    z = x @ w.T
    dz = eps_of(x.shape[1]) * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
        dz = dz + 2.0 ** -23 * np.abs(z)
    y = act(z, kind)
    err = SLOPE_MAX * dz + (0.0 if kind == "none" else ACT * np.abs(y) + TINY)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
        err = err + 2.0 ** -23 * np.abs(y)
    return (y, _rounded(y, err)), (z, _rounded(z, dz))


def linear_act_bwd(z, d_y, w, kind):
    """((d_x, bound), (d_z, bound), (d_bias, bound))."""
    d_y = np.asarray(d_y, np.float64)
    if kind == "none":
        d_z, e = d_y, np.zeros_like(d_y)
        b = e   # d_z is d_y itself
    else:
        d_z = d_y * slope(z, kind)
        e = ACT * np.abs(d_y) + 2.0 ** -23 * np.abs(d_z)
        b = _rounded(d_z, e)
    d_b = d_z.sum(0)
    b_b = e.sum(0) + (d_y.shape[0] + 8) * 2.0 ** -24 * np.abs(d_z).sum(0) + 2.0 ** -23 * np.abs(d_b)
    return _product(d_z, b, w), (d_z, b), (d_b, b_b)


def distill(logits, indices, teacher, temperature, d_loss=None, lse_in=None):
    """((loss, bound), (lse, bound), (d_logits, bound) or None)."""
    z = np.asarray(logits, np.float64) / temperature
    idx = np.asarray(indices)
    V = z.shape[1]
    valid = (idx >= 0) & (idx < V)
    t = np.where(valid, np.asarray(teacher, np.float64), -np.inf) / temperature
    top = t.max(1, keepdims=True)
    has = np.isfinite(top[:, 0])
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(t - top)
    total = np.where(has, e.sum(1), 1.0)[:, None]
    q = e / total
    with np.errstate(divide="ignore"):
        log_q = t - top - np.log(total)
    m = z.max(1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(z - m).sum(1))
    zi = np.take_along_axis(z, np.where(valid, idx, 0), 1)
    with np.errstate(invalid="ignore"):
        terms = np.where(q > 0, q * (log_q - zi + lse[:, None]), 0.0)
    loss = temperature ** 2 * terms.sum(1) * has
    # fp32 steps: quotients by T and differences of the values below (each at
    # most 2^-22 of the largest), the exponential sum (2^-20 relative with its
    # arguments), logarithms and the sum over k
    size = 1.0 + np.where(np.isfinite(z), np.abs(z), 0).max(1) + np.where(np.isfinite(t), np.abs(t), 0).max(1)
    b_lse = 2.0 ** -20 * size
    b_loss = temperature ** 2 * 2.0 ** -19 * size
    grad = None
    if d_loss is not None:
        ref = lse if lse_in is None else np.asarray(lse_in, np.float64)
        p = np.exp(z - ref[:, None])
        qs = np.zeros_like(z)
        for row in range(z.shape[0]):
            np.add.at(qs[row], idx[row][valid[row]], q[row][valid[row]])
        coef = np.asarray(d_loss, np.float64)[:, None] * temperature
        d = np.where(has[:, None], coef * (p - qs), 0.0)
        # p and q carry the absolute error of their exponents (2^-21 of the values above)
        b = _rounded(d, np.abs(coef) * (p + qs) * 2.0 ** -19 * size[:, None])
        grad = (d, b)
    return (loss, b_loss), (lse, b_lse), grad


def distill_spread(logits, indices, teacher, temperature, d_loss=None, lse_in=None, two=False):
    """As ``distill``, with bounds that go by how far the logits of a row are from each other, not from zero: what a
    row has in common cancels in p and in the loss, and every value that an output is made of is held against the
    row's own maximum.  (The gradient from a saved ``lse_in`` is that of ``lse_in`` as it was saved.)

    In units of 2^-24, with s = |z - max| / T (s_t for the teacher) and S = sum p s:
      an exponent (z - max) c: 3 s for c = fp32(fp32(1/T) fp32(log2 e)), s for its own rounding, s for each of at
      most three changes of maximum (tile, warp, CTA): 8 s of a weight with some to spare, 8 S of their sum;
      a weight's exponential 4, each change of maximum 4 + 1; a sum over V: V / 256 additions in a row in one thread
      and 5 for a change of maximum per tile of 8192, then 16 over lanes, warps and CTAs: V / 200 + 128 with some to
      spare;
      the teacher's weights: the same over at most 8 additions in a thread, 128;
      1 / sum, the products with coef and the difference p - q: 8, within the 128.
    A logarithm adds 2 of itself, a quotient by T and a sum 2 of theirs each.  From a saved lse the exponent is
    z / T - lse: 8 of its size, and while |lse| < 64 another 8 of |z| / T + |lse|.  ``two``: a step of two launches,
    whose second takes a row with |lse| < 64 from the lse of the first: 2 of |z| / T, 3 of |lse| with its own
    rounding and one of log V <= 15, altogether within 4 (|z| / T + |lse| + 4).
    """
    (loss, _), (lse, _), grad = distill(logits, indices, teacher, temperature, d_loss, lse_in)
    unit = 2.0 ** -24
    z = np.asarray(logits, np.float64) / temperature
    idx = np.asarray(indices)
    V = z.shape[1]
    valid = (idx >= 0) & (idx < V)
    t = np.where(valid, np.asarray(teacher, np.float64), -np.inf) / temperature
    far = lambda a: np.where(np.isfinite(a), np.abs(a), 0.0)   # noqa: E731  (a weight of zero: no matter how far)
    m = z.max(1, keepdims=True)
    s = far(z - m)
    p = np.exp(z - m)
    p /= p.sum(1, keepdims=True)
    top = t.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    s_t = far(t - top)
    q = np.exp(t - top)
    total = q.sum(1, keepdims=True)
    q = q / np.where(total > 0, total, 1.0)
    S, S_t = (p * s).sum(1, keepdims=True), (q * s_t).sum(1, keepdims=True)
    of_sum = (V / 200 + 128 + 8 * S) * unit
    of_q = (128 + 8 * (s_t + S_t)) * unit
    log_s = lse[:, None] - m
    at = far(np.take_along_axis(z, np.where(valid, idx, 0), 1) - m)
    log_total = np.log(np.where(total > 0, total, 1.0))
    parts = s_t + np.abs(log_total) + at + np.abs(log_s)        # what a term of the loss is added from
    b_loss = temperature ** 2 * ((q * (of_q * parts + 8 * unit * parts)).sum(1) + of_sum[:, 0] + 128 * unit)
    b_lse = of_sum[:, 0] + unit * (2 * np.abs(log_s[:, 0]) + 2 * np.abs(m[:, 0]) + np.abs(lse))
    if grad is None:
        return (loss, b_loss), (lse, b_lse), None
    d = grad[0]
    if lse_in is None:
        of_p = of_sum + 8 * s * unit
        if two:
            of_p = of_p + np.where(np.abs(lse[:, None]) < 64, 4 * (far(z) + np.abs(lse[:, None]) + 4), 0.0) * unit
    else:
        ref = np.asarray(lse_in, np.float64)[:, None]
        p = np.exp(z - ref)
        near = np.where(np.abs(ref) < 64, far(z) + np.abs(ref), 0.0)
        of_p = (16 + 8 * far(z - ref) + 8 * near) * unit
    coef = np.abs(np.asarray(d_loss, np.float64)[:, None] * temperature)
    err = p * of_p
    for row in range(z.shape[0]):
        np.add.at(err[row], idx[row][valid[row]], (q * of_q)[row][valid[row]])
    return (loss, b_loss), (lse, b_lse), (d, _rounded(d, coef * err))
