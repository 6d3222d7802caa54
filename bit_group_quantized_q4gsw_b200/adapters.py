"""The operators of include/q4gsw_adapters.h on torch tensors: many low-rank
adapters on one frozen base, the norms around a block, and the norm and clip of a
list of gradients.

Argument marshalling only, as in layer.py, whose checks these calls share.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .binding import _check, library
from .layer import _blob, _call, _empty, _f16, _f32, _i32, _need, _rows, _u8

_like = {}   # an empty tensor of each type and device: new tensors of its kind cost less than torch.empty


def _new(shape, dtype, index: int):
    t = _like.get((dtype, index))
    if t is None:
        t = _like[dtype, index] = _empty(0, dtype=dtype, device=index)
    return t.new_empty(shape)


def _out(t, name: str, dtype, shape, index: int):
    """(tensor, pointer) of an output: the caller's buffer, or a new one."""
    if t is None:
        t = _new(shape, dtype, index)
        return t, t.data_ptr()
    return t, _need(t, name, dtype, shape, index)


_plan_bytes = {}   # bytes of a plan by (M, L): a pure function of these


def _plan_size(M: int, L: int) -> int:
    n = _plan_bytes.get((M, L))
    if n is None:
        n = int(library().q4gsw_adapters_plan_bytes(M, L))
        if len(_plan_bytes) < 4096:
            _plan_bytes[M, L] = n
    return n


def q4gsw_adapters_plan(ids, L: int, plan=None):
    """The plan of a batch: ids int32 [M], each token's adapter of L, or -1 for none -> an int32 tensor for
    q4gsw_adapters_fwd and _bwd.  One plan serves every projection of every layer that the batch goes through."""
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dim() != 1:
        raise ValueError(f"ids must have 1 dim (got {ids.dim()})")
    M, index = ids.shape[0], ids.get_device()
    pi = _need(ids, "ids", _i32, (M,), index)
    nbytes = _plan_size(M, L)
    if plan is None:
        plan = _new(max(nbytes // 4, 4), _i32, index)
    pp, words = _sized(plan, "plan", _i32, index)
    _call("q4gsw_adapters_plan", index, pi, M, L, pp, 4 * words)
    return plan


def _sized(t, name: str, dtype, index: int):
    """(pointer, elements) of a caller's buffer of any size."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return _need(t, name, dtype, (t.numel(),), index), t.numel()


def _adapters(plan, a, b, scale, M: int, N: int, K: int, index: int):
    """(L, r) and the pointers of the plan, the adapters and their factors."""
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("a must be a float16 tensor of 3 dims, [L, r, K]")
    L, r = a.shape[0], a.shape[1]
    pa = _need(a, "a", _f16, (L, r, K), index)
    pb = _need(b, "b", _f16, (L, N, r), index)
    ps = None if scale is None else _need(scale, "scale", _f32, (L,), index)
    if not isinstance(plan, torch.Tensor) or plan.dtype is not _i32:
        raise TypeError("plan must be the int32 tensor of q4gsw_adapters_plan")
    if plan.get_device() != index or not plan.is_contiguous():
        raise ValueError(f"plan must be contiguous and on cuda:{index}")
    if 4 * plan.numel() < _plan_size(M, L):
        raise ValueError(f"plan holds {4 * plan.numel()} bytes, {M} tokens over {L} adapters need {_plan_size(M, L)}")
    return L, r, plan.data_ptr(), pa, pb, ps


def q4gsw_adapters_fwd(packed, N: int, K: int, group_size: int, plan, a, b, x, scale=None, bias=None, residual=None,
                       y=None, u=None, save_u: bool = False, f32s: bool = False):
    """y = x W^T + bias + residual + s_a (x A_a^T) B_a^T with a each token's own adapter: x fp16 [M, K], a fp16
    [L, r, K], b fp16 [L, N, r], scale fp32 [L] -> y fp16 [M, N] (which may be the residual's buffer).  `plan`
    is q4gsw_adapters_plan of the batch's ids and L.  With save_u (or a u buffer) returns (y, u), u fp32 [M, r]
    the low-rank intermediate that the backward pass reads."""
    px, M, index = _rows(x, "x", _f16, K)
    pw = _blob(packed, N, K, group_size, f32s, index)
    L, r, pp, pa, pb, ps = _adapters(plan, a, b, scale, M, N, K, index)
    pbias = None if bias is None else _need(bias, "bias", _f16, (N,), index)
    pr = None if residual is None else _need(residual, "residual", _f16, (M, N), index)
    give = save_u or u is not None
    y, py = _out(y, "y", _f16, (M, N), index)
    if py == px and M:
        raise ValueError("y must not be x's buffer")
    u, pu = _out(u, "u", _f32, (M, r), index)
    _call("q4gsw_adapters_fwd_f32s" if f32s else "q4gsw_adapters_fwd", index, pw, N, K, group_size, pp, pa, pb, ps, L, r,
          px, M, pbias, pr, py, pu)
    return (y, u) if give else y


def q4gsw_adapters_bwd(packed, N: int, K: int, group_size: int, plan, a, b, x, u, d_y, scale=None, d_x=None, d_a=None,
                       d_b=None, v=None, want_x: bool = True, want_adapters: bool = True, accumulate: bool = False,
                       f32s: bool = False):
    """(d_x fp16 [M, K], d_a fp32 [L, r, K], d_b fp32 [L, N, r]) from x and u of the forward and d_y fp16 [M, N].
    Without want_x d_x is None, without want_adapters d_a and d_b are (x and u may then be None).  With
    accumulate the adapters' gradients are added to what the buffers d_a and d_b hold."""
    pd, M, index = _rows(d_y, "d_y", _f16, N)
    pw = _blob(packed, N, K, group_size, f32s, index)
    L, r, pp, pa, pb, ps = _adapters(plan, a, b, scale, M, N, K, index)
    px = pu = pdx = pda = pdb = None
    want_x = want_x or d_x is not None
    if want_x:
        d_x, pdx = _out(d_x, "d_x", _f16, (M, K), index)
    if want_adapters or d_a is not None or d_b is not None:
        if accumulate and (d_a is None or d_b is None):
            raise ValueError("accumulate needs the buffers d_a and d_b")
        px = _need(x, "x", _f16, (M, K), index)
        pu = _need(u, "u", _f32, (M, r), index)
        d_a, pda = _out(d_a, "d_a", _f32, (L, r, K), index)
        d_b, pdb = _out(d_b, "d_b", _f32, (L, N, r), index)
    v, pv = _out(v, "v", _f32, (M, r), index)
    if M and (pdx == pd or (pda and (pdx == px or pv == pu))):
        raise ValueError("d_x must not be d_y's or x's buffer, nor v u's")
    _call("q4gsw_adapters_bwd_f32s" if f32s else "q4gsw_adapters_bwd", index, pw, N, K, group_size, pp, pa, pb, ps, L, r,
          px, pu, pd, M, int(accumulate), pv, pdx, pda, pdb)
    return d_x, d_a, d_b


def _out_like(t, name: str, like, index: int):
    """The same for a tensor of another's type and shape (known to be contiguous)."""
    if t is None:
        t = torch.empty_like(like)
        return t, t.data_ptr()
    return t, _need(t, name, like.dtype, like.shape, index)


def _norm_operands(M: int, D: int, index: int, block, w_post, gate, w_pre):
    pblock = ppost = pgate = ppre = None
    rows = 0
    if block is not None:
        pblock = _need(block, "block", _f16, (M, D), index)
        if w_post is not None:
            ppost = _need(w_post, "w_post", _f16, (D,), index)
        if gate is not None:
            rows = int(isinstance(gate, torch.Tensor) and gate.dim() == 2)
            pgate = _need(gate, "gate", _f16, (M, D) if rows else (D,), index)
    elif w_post is not None or gate is not None:
        raise ValueError("without a block there is no w_post and no gate")
    if w_pre is not None:
        ppre = _need(w_pre, "w_pre", _f16, (D,), index)
    return pblock, ppost, pgate, rows, ppre


def q4gsw_norms_fwd(h, block=None, w_post=None, gate=None, residual_scale: float = 1.0, w_pre=None, eps: float = 1e-6,
                    weight_offset: float = 0.0, h_out=None, x=None):
    """(x, h') between two blocks: n = RMS norm of `block` with w_post (block itself without w_post),
    h' = residual_scale h + gate n, x = RMS norm of h' with w_pre; weights are weight_offset + w.  h, block fp16
    [M, D], w_post, w_pre fp16 [D], gate fp16 [D] or [M, D].  h_out may be h's own buffer.  Without a block h' is
    residual_scale h, and h itself where that is 1 and no buffer is given; without w_pre x is None."""
    if not isinstance(h, torch.Tensor) or h.dim() != 2:
        raise ValueError("h must be a float16 tensor of 2 dims")
    (M, D), index = h.shape, h.get_device()
    ph = _need(h, "h", _f16, (M, D), index)
    pblock, ppost, pgate, rows, ppre = _norm_operands(M, D, index, block, w_post, gate, w_pre)
    po = px = None
    if block is None and residual_scale == 1.0 and h_out is None:
        if w_pre is None:
            raise ValueError("without a block and w_pre there is nothing to compute")
        h_out = h
    else:
        h_out, po = _out_like(h_out, "h_out", h, index)
    if w_pre is not None:
        x, px = _out_like(x, "x", h, index)
    elif x is not None:
        raise ValueError("x needs w_pre")
    _call("q4gsw_norms_fwd", index, ph, pblock, ppost, pgate, rows, residual_scale, ppre, weight_offset, eps, M, D, po, px)
    return x, h_out


class NormsGrad(NamedTuple):
    """Gradients of q4gsw_norms_bwd; None where there is no such input or it was not asked for."""
    residual: torch.Tensor          # fp16 [M, D], of h
    block: torch.Tensor | None      # fp16 [M, D]
    gate: torch.Tensor | None       # fp16 [M, D] with a gate for every row, else fp32 [D]
    w_post: torch.Tensor | None     # fp32 [D]
    w_pre: torch.Tensor | None      # fp32 [D]


_norms_bytes = {}   # workspace bytes by (M, D)


def q4gsw_norms_bwd(h_out, d_x=None, d_h=None, block=None, w_post=None, gate=None, residual_scale: float = 1.0,
                    w_pre=None, eps: float = 1e-6, weight_offset: float = 0.0, want_weights: bool = False,
                    d_residual=None, d_block=None, d_gate=None, d_w_post=None, d_w_pre=None, workspace=None):
    """NormsGrad from d_x fp16 [M, D], the gradient of x (with w_pre and h_out as the forward wrote it; h_out may be
    None without), and d_h fp16 [M, D], what reaches h' from later layers.  A gate for every row always has its
    gradient; the sums over the rows (both weights, one gate for all rows) are computed with want_weights or where
    a buffer is given."""
    d = d_x if d_x is not None else d_h
    if not isinstance(d, torch.Tensor) or d.dim() != 2:
        raise ValueError("d_x or d_h must be a float16 tensor of 2 dims")
    (M, D), index = d.shape, d.get_device()
    p = _need(d, "d_x" if d_x is not None else "d_h", _f16, (M, D), index)
    if (d_x is None) != (w_pre is None):
        raise ValueError("d_x and w_pre go together")
    pblock, ppost, pgate, rows, ppre = _norm_operands(M, D, index, block, w_post, gate, w_pre)
    pdx = None if d_x is None else p
    ph = None if d_x is None else _need(h_out, "h_out", _f16, (M, D), index)
    pdh = None if d_h is None else p if d_h is d else _need(d_h, "d_h", _f16, (M, D), index)
    if (d_block is not None and block is None) or (d_gate is not None and gate is None) or \
            (d_w_post is not None and w_post is None) or (d_w_pre is not None and w_pre is None):
        raise ValueError("d_block, d_gate, d_w_post and d_w_pre are gradients of inputs that are there")
    d_residual, pr = _out_like(d_residual, "d_residual", d, index)
    pdb = pgr = pg = pwo = pwe = pws = None
    nbytes = 0
    if block is not None:
        d_block, pdb = _out_like(d_block, "d_block", d, index)
    if rows:
        d_gate, pgr = _out_like(d_gate, "d_gate", d, index)
    if want_weights or d_gate is not None or d_w_post is not None or d_w_pre is not None:
        # the sums; one allocation for those that have no buffer
        feature = gate is not None and not rows
        new = want_weights and [t is None and there for t, there in (
            (d_gate, feature), (d_w_post, w_post is not None), (d_w_pre, w_pre is not None))]
        if new and any(new):
            sums = _new((sum(new), D), _f32, index)
            at, views = sums.data_ptr(), sums.unbind()
            k = 0
            if new[0]:
                d_gate, pg, k = views[0], at, 1
            if new[1]:
                d_w_post, pwo, k = views[k], at + 4 * D * k, k + 1
            if new[2]:
                d_w_pre, pwe = views[k], at + 4 * D * k
        if pg is None and feature and d_gate is not None:
            pg = _need(d_gate, "d_gate", _f32, (D,), index)
        if pwo is None and d_w_post is not None:
            pwo = _need(d_w_post, "d_w_post", _f32, (D,), index)
        if pwe is None and d_w_pre is not None:
            pwe = _need(d_w_pre, "d_w_pre", _f32, (D,), index)
    if pg or pwo or pwe:
        need = _norms_bytes.get((M, D))
        if need is None:
            need = int(library().q4gsw_norms_workspace_bytes(M, D))
            if len(_norms_bytes) < 4096:
                _norms_bytes[M, D] = need
        if workspace is None:
            nbytes = max(need, 16)
            workspace = _new(nbytes, _u8, index)
            pws = workspace.data_ptr()
        else:
            pws, nbytes = _sized(workspace, "workspace", _u8, index)
    _call("q4gsw_norms_bwd", index, ph, pdx, pdh, pblock, ppost, pgate, rows, residual_scale, ppre, weight_offset, eps, M,
          D, pr, pdb, pgr, pwe, pwo, pg, pws, nbytes)
    return NormsGrad(d_residual, d_block, d_gate, d_w_post, d_w_pre)


class GradSet:
    """A list of gradient buffers (and what their clipped values go to) for q4gsw_grad_norm and q4gsw_grad_clip.
    Holds the tensors, and their table on the device: made once for buffers that a program keeps from step to step."""

    def __init__(self, grads, outs, table, index: int):
        self.grads, self.outs, self.table, self.index = grads, outs, table, index
        # the table has addresses: the storages live as long as it, also where a tensor is given another one
        self._storages = [t.detach() for t in grads] + ([] if outs is grads else [t.detach() for t in outs])
        self.table_bytes, self.table_ptr = table.numel(), table.data_ptr()
        self.long = self.table_bytes > 64 * 32      # records of 32 bytes; up to 64 need no workspace


def _elements(t, name: str, index: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dtype not in (_f32, _f16):
        raise TypeError(f"{name} must be float32 or float16 (got {t.dtype})")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), t.numel(), int(t.dtype is _f16)


def q4gsw_grad_set(grads, outs=None) -> GradSet:
    """A GradSet of gradients (fp32 or fp16 tensors of one device, any shapes).  `outs`, one tensor of as many elements
    for each gradient, fp32 or fp16, receive the clipped values; without them the gradients are clipped in place, and
    must not overlap one another, also where only their norm is asked for.

    Make it once for buffers that stay where they are: it fills a record of 32 bytes for every 1024 elements on the
    host (2 ms for 200 million elements, where a clip takes 0.1), copies them and waits for the current stream.  With
    gradients that are allocated anew each step (zero_grad(set_to_none=True)) that is paid each step: keep the
    buffers, or have their sums accumulated in them (set_to_none=False)."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    first = grads[0]
    index = first.get_device() if isinstance(first, torch.Tensor) and first.device.type == "cuda" else -1
    src = [_elements(g, f"grads[{i}]", index) for i, g in enumerate(grads)]
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} outs for {len(grads)} gradients")
    dst = src if outs is grads else [_elements(o, f"outs[{i}]", index) for i, o in enumerate(outs)]
    spans = []
    for i, (s, d) in enumerate(zip(src, dst)):
        if s[1] != d[1]:
            raise ValueError(f"outs[{i}] has {d[1]} elements, its gradient {s[1]}")
        if s[1]:
            spans.append((d[0], d[0] + d[1] * (2 if d[2] else 4), i))
            if s[0] != d[0] or s[2] != d[2]:
                spans.append((s[0], s[0] + s[1] * (2 if s[2] else 4), -1))
    # an out must not overlap another out or a gradient that is not its own
    any_end = out_end = -1
    for lo, hi, i in sorted(spans):
        if lo < (any_end if i >= 0 else out_end):
            raise ValueError("outs overlap each other or another gradient")
        any_end = max(any_end, hi)
        if i >= 0:
            out_end = max(out_end, hi)
    n = len(grads)
    ptrs, i32, i64 = ctypes.c_void_p * n, ctypes.c_int * n, ctypes.c_int64 * n
    sizes = i64(*(s[1] for s in src))
    lib = library()
    nbytes = int(lib.q4gsw_grad_table_bytes(n, sizes))
    host = torch.empty(max(nbytes, 1), dtype=_u8)
    _check("q4gsw_grad_table",
           lib.q4gsw_grad_table(n, ptrs(*(s[0] for s in src)), i32(*(s[2] for s in src)), ptrs(*(d[0] for d in dst)),
                                i32(*(d[2] for d in dst)), sizes, host.data_ptr(), host.numel()))
    table = host.to(first.device)
    torch.cuda.current_stream(first.device).synchronize()     # the set may be used on any stream
    return GradSet(grads, outs, table, index)


_grad_bytes = None   # of a workspace


def _grad_call(name: str, grads: GradSet, head, norm, workspace):
    global _grad_bytes
    if not isinstance(grads, GradSet):
        raise TypeError("grads must be a GradSet (q4gsw_grad_set)")
    norm, pn = _out(norm, "norm", _f32, (1,), grads.index)
    pw, nbytes = None, 0
    if workspace is not None:
        pw, nbytes = _sized(workspace, "workspace", _u8, grads.index)
    elif grads.long:
        if _grad_bytes is None:
            _grad_bytes = int(library().q4gsw_grad_workspace_bytes())
        workspace, nbytes = _new(_grad_bytes, _u8, grads.index), _grad_bytes
        pw = workspace.data_ptr()
    _call(name, grads.index, grads.table_ptr, grads.table_bytes, *head, pn, pw, nbytes)
    return norm


def q4gsw_grad_norm(grads: GradSet, inv_scale: float = 1.0, norm=None, workspace=None):
    """norm fp32 [1] = |inv_scale| sqrt(sum of the squares of every gradient of the set)."""
    return _grad_call("q4gsw_grad_norm", grads, (inv_scale,), norm, workspace)


def q4gsw_grad_clip(grads: GradSet, max_norm: float, inv_scale: float = 1.0, norm=None, workspace=None):
    """Writes inv_scale min(1, max_norm / (norm + 1e-6)) g to every gradient's out, and returns the norm, fp32 [1]."""
    return _grad_call("q4gsw_grad_clip", grads, (max_norm, inv_scale), norm, workspace)
