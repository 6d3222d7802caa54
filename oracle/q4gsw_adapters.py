"""Plain CPU oracle for the adapters of many requests, the norms around a block
and the norm and clip of a list of gradients.

TEST INFRASTRUCTURE ONLY, under the same rule as ``q4gsw_oracle``.  Everything is
computed in fp64 from the definitions.  Functions return (value, bound) pairs; a
bound counts the roundings of the kernels' arithmetic:

  acc(n)  sums of n products in fp32 on the tensor cores or in registers: at most
          2^-23 of the absolute products a step (the tensor cores truncate), and
          not less than 64 steps;
  SPLIT   2^-23 of the largest value of a token's row (in sums over ranks) or of a rank's
          column (over tokens): the two fp16 parts of the intermediate over a power of
          two with that value in [1, 2).  The first part is off by at most half a step,
          2^-11, and the second, the rest, by half a step of a value below 2^-11: 2^-23;
  SCALED  2^-21 relative: the products and the scaling back;
  STAT    2^-18 relative: a norm's factor.  At most 32 terms a thread, 5 shuffles
          and 32 warps are 69 roundings of 2^-24 in the sum of squares, half of
          that in its root, rsqrtf's 2^-22 and four products;
  HALF, TINY  one rounding to fp16, as in ``q4gsw_layer``.
"""
from __future__ import annotations

import math

import numpy as np

from .q4gsw_layer import HALF, TINY, _rounded, eps_of

SPLIT = 2.0 ** -23
SCALED = 2.0 ** -21
STAT = 2.0 ** -18


def acc(n: int) -> float:
    return max(n, 64) * 2.0 ** -23


def _factors(scale, L):
    return np.ones(L) if scale is None else np.asarray(scale, np.float64)


def _low(ids, q, b_q, mat, scale):
    """(f q mat, bound) per token; mat [L, r, C], rows without an adapter zero."""
    out, err = np.zeros((len(ids), mat.shape[2])), np.zeros((len(ids), mat.shape[2]))
    f = _factors(scale, mat.shape[0])
    for a in np.unique(ids):
        if a < 0:
            continue
        at, m = ids == a, np.asarray(mat[a], np.float64)
        am = np.abs(m)
        top = np.abs(q[at]).max(1, keepdims=True)
        out[at] = f[a] * (q[at] @ m)
        err[at] = abs(f[a]) * (b_q[at] @ am + SPLIT * top * am.sum(0) + acc(0) * (np.abs(q[at]) @ am))
    return out, err


def _down(ids, act, mat, scale):
    """(f act mat^T, bound) per token; mat [L, r, C]."""
    out, err = np.zeros((len(ids), mat.shape[1])), np.zeros((len(ids), mat.shape[1]))
    f = _factors(scale, mat.shape[0])
    for a in np.unique(ids):
        if a < 0:
            continue
        at, m = ids == a, np.asarray(mat[a], np.float64)
        out[at] = f[a] * (act[at] @ m.T)
        err[at] = abs(f[a]) * acc(m.shape[1]) * (np.abs(act[at]) @ np.abs(m).T)
    return out, err


def adapters_fwd(x, w, ids, a, b, scale=None, bias=None, residual=None):
    """((y, bound), (u, bound)): x [M, K], w [N, K] dequantised, a [L, r, K], b [L, N, r]."""
    x, ids = np.asarray(x, np.float64), np.asarray(ids)
    u, b_u = _down(ids, x, a, None)
    d, e = _low(ids, u, b_u, np.transpose(b, (0, 2, 1)), scale)
    if residual is not None:
        d = d + np.asarray(residual, np.float64)
        e = e + 2.0 ** -23 * np.abs(d)
    low = _rounded(d, e)                       # the term in the output's place, fp16
    base = x @ w.T
    if bias is not None:
        base = base + np.asarray(bias, np.float64)
    y = base + d
    err = eps_of(x.shape[1]) * (np.abs(x) @ np.abs(w).T) + low + 2.0 ** -22 * (np.abs(base) + np.abs(d))
    return (y, _rounded(y, err)), (u, b_u)


def adapters_bwd(x, u, d_y, w, ids, a, b, scale=None):
    """((d_x, bound), (d_a, bound), (d_b, bound)) from u as the forward saved it."""
    x, u, d_y = (np.asarray(v, np.float64) for v in (x, u, d_y))
    ids = np.asarray(ids)
    L, r, K = a.shape
    f = _factors(scale, L)
    v, b_v = _down(ids, d_y, np.transpose(b, (0, 2, 1)), scale)
    low, e = _low(ids, v, b_v, np.asarray(a), None)
    low_b = _rounded(low, e)
    base = d_y @ w
    d_x = base + low
    err = eps_of(w.shape[0]) * (np.abs(d_y) @ np.abs(w)) + low_b + 2.0 ** -22 * (np.abs(base) + np.abs(low))
    d_a, e_a = np.zeros(a.shape), np.zeros(a.shape)
    d_b, e_b = np.zeros(b.shape), np.zeros(b.shape)
    for i in range(L):
        at = ids == i
        n = int(at.sum())
        if not n:
            continue
        d_a[i] = v[at].T @ x[at]
        top_v, top_u = (np.abs(v[at]) + b_v[at]).max(0), np.abs(u[at]).max(0)
        e_a[i] = SPLIT * np.outer(top_v, np.abs(x[at]).sum(0))
        e_a[i] += b_v[at].T @ np.abs(x[at]) + (SCALED + acc(n)) * ((np.abs(v[at]) + b_v[at]).T @ np.abs(x[at]))
        d_b[i] = f[i] * (d_y[at].T @ u[at])
        e_b[i] = abs(f[i]) * SPLIT * np.outer(np.abs(d_y[at]).sum(0), top_u)
        e_b[i] += abs(f[i]) * (SCALED + acc(n)) * (np.abs(d_y[at]).T @ np.abs(u[at]))
    return (d_x, _rounded(d_x, err)), (d_a, e_a), (d_b, e_b)


def plan(ids, L):
    """(order, first): the tokens sorted by adapter, those without one (or with an id outside [0, L)) last, and
    where each adapter starts."""
    g = [i if 0 <= i < L else L for i in ids]
    order = sorted(range(len(g)), key=lambda m: g[m])        # a stable sort
    return order, [sum(v < i for v in g) for i in range(L + 2)]


# ---------------------------------------------------------------- norms
def _norm(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def _opt(v):
    return None if v is None else np.asarray(v, np.float64)


def _stream(h, block, w_post, gate, f, offset, eps):
    """(h', error, n, error of n)."""
    h, block, w_post, gate = (_opt(v) for v in (h, block, w_post, gate))
    s = f * h
    if block is None:
        return s, 2.0 ** -24 * np.abs(s), None, None
    n, e_n = block, np.zeros_like(block)
    if w_post is not None:
        n = block * _norm(block, eps) * (offset + w_post)
        e_n = STAT * np.abs(n) + 2.0 ** -23 * np.abs(block * _norm(block, eps)) * (abs(offset) + np.abs(w_post))
    g = np.ones(1) if gate is None else gate
    out = s + g * n
    return out, np.abs(g) * e_n + 2.0 ** -22 * (np.abs(s) + np.abs(g * n)), n, e_n


def norms_fwd(h, block=None, w_post=None, gate=None, residual_scale=1.0, w_pre=None, eps=1e-6, weight_offset=0.0):
    """((x, bound) or None, (h', bound))."""
    s, e, _, _ = _stream(h, block, w_post, gate, residual_scale, weight_offset, eps)
    x = None
    if w_pre is not None:
        w = np.asarray(w_pre, np.float64)
        k = _norm(s, eps)
        far = np.sqrt((e * e).sum(1, keepdims=True) / np.maximum((s * s).sum(1, keepdims=True), 1e-300))
        v = s * k * (weight_offset + w)
        b = k * np.abs(weight_offset + w) * e + np.abs(v) * (STAT + far)
        b = b + 2.0 ** -23 * np.abs(s * k) * (abs(weight_offset) + np.abs(w))
        x = (v, _rounded(v, b))
    return x, (s, _rounded(s, e))


def _slope(v, w, aw, d, e_d, eps):
    """(gradient of v through v norm(v) w, error): aw the absolute value of w's terms, e_d the error of d."""
    k = _norm(v, eps)
    e = d * w
    mean, size = (e * v).mean(1, keepdims=True), (np.abs(d) * aw * np.abs(v)).mean(1, keepdims=True)
    out = k * e - v * k ** 3 * mean
    b = k * (STAT * np.abs(e) + 2.0 ** -22 * np.abs(d) * aw + e_d * aw)
    b = b + np.abs(v) * k ** 3 * (3 * STAT * np.abs(mean) + 2 * STAT * size + (e_d * aw * np.abs(v)).mean(1, keepdims=True))
    return out, b + 2.0 ** -22 * (k * np.abs(e) + np.abs(v) * k ** 3 * np.abs(mean))


def norms_bwd(h_out, d_x=None, d_h=None, block=None, w_post=None, gate=None, residual_scale=1.0, w_pre=None, eps=1e-6,
              weight_offset=0.0):
    """Dict of (value, bound): residual, and where there are such inputs block, gate (rows or their sum), w_post, w_pre."""
    h_out, d_x, d_h, block, w_post, gate, w_pre = (_opt(v) for v in (h_out, d_x, d_h, block, w_post, gate, w_pre))
    rows = (d_x if d_x is not None else d_h).shape[0]
    out = {}

    def total(v, e):
        return v.sum(0), e.sum(0) + (rows + 16) * 2.0 ** -24 * np.abs(v).sum(0)

    d = np.zeros((rows, (d_x if d_x is not None else d_h).shape[1])) if d_h is None else d_h
    e = np.zeros_like(d)
    if d_x is not None:
        w, aw = weight_offset + w_pre, abs(weight_offset) + np.abs(w_pre)
        g, e_g = _slope(h_out, w, aw, d_x, np.zeros_like(d_x), eps)
        term = d_x * h_out * _norm(h_out, eps)
        out["w_pre"] = total(term, 2 * STAT * np.abs(term))
        e = e_g + 2.0 ** -23 * (np.abs(d) + np.abs(g))
        d = d + g
    r = residual_scale * d
    out["residual"] = (r, _rounded(r, abs(residual_scale) * e + 2.0 ** -24 * np.abs(r)))
    if block is None:
        return out
    _, _, n, e_n = _stream(np.zeros_like(d), block, w_post, None, 0.0, weight_offset, eps)
    p, e_p = d, e
    if gate is not None:
        t = d * n
        e_t = e * np.abs(n) + (np.abs(d) + e) * e_n + 2.0 ** -22 * np.abs(t)
        out["gate"] = (t, _rounded(t, e_t)) if gate.ndim == 2 else total(t, e_t)
        p, e_p = d * gate, e * np.abs(gate) + 2.0 ** -24 * np.abs(d * gate)
    if w_post is not None:
        term = p * block * _norm(block, eps)
        out["w_post"] = total(term, 2 * STAT * np.abs(term) + e_p * np.abs(block * _norm(block, eps)))
        p, e_p = _slope(block, weight_offset + w_post, abs(weight_offset) + np.abs(w_post), p, e_p, eps)
    out["block"] = (p, _rounded(p, e_p))
    return out


# ---------------------------------------------------------------- gradient lists
def grad_norm(grads, inv_scale=1.0):
    """(norm, bound): fp64 sums, one rounding to fp32 (half a step of 2^-149 where the norm is subnormal)."""
    n = abs(inv_scale) * math.sqrt(math.fsum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    return n, 2.0 ** -23 * n + 2.0 ** -150


def grad_clip(grads, max_norm, inv_scale=1.0, half=False):
    """[(out, bound)]: the factor is off by at most four roundings of 2^-24."""
    n, _ = grad_norm(grads, inv_scale)
    k = inv_scale * min(1.0, max_norm / (n + 1e-6))
    res = []
    for g in grads:
        v = np.asarray(g, np.float64) * k
        e = 6 * 2.0 ** -24 * np.abs(v) + 2.0 ** -149
        res.append((v, _rounded(v, e) if half else e))
    return res
