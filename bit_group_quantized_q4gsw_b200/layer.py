"""The operators of include/q4gsw_layer.h on torch tensors: the gated
feed-forward block, the projection with an epilogue and the distillation loss.

Argument marshalling only, as in binding.py.  Besides dtype, contiguity and
device every shape is checked here, since the C calls see pointers alone.  The
calls run on the current stream of the tensors' device, whichever device is
current.  A decode call takes a few microseconds on the GPU, so the checks are
written to cost about as little: one test of everything per tensor, and words
only where it fails.
"""
from __future__ import annotations

import torch

from .binding import _check, library

ACTS = {"none": 0, "silu": 1, "gelu_tanh": 2}
_GATED = {"silu": 1, "gelu_tanh": 2}

# the current stream's handle and device without building Python objects; None in a build without CUDA
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_now = getattr(torch._C, "_cuda_getDevice", None)

_f16, _f32, _i32, _u8 = torch.float16, torch.float32, torch.int32, torch.uint8
_empty = torch.empty


def _refuse(t, name: str, dtype, shape, index: int):
    """Why a tensor is not what a call needs."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")
    raise ValueError(f"{name} must be contiguous")


def _need(t, name: str, dtype, shape, index: int):
    """The pointer of a tensor of this type and shape on CUDA device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _rows(t, name: str, dtype, cols: int):
    """(pointer, rows, device index) of the [rows, cols] tensor that fixes the batch and the device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims (got {t.dim()})")
    n, index = t.shape[0], t.get_device()
    return _need(t, name, dtype, (n, cols), index), n, index


_blob_bytes = {}   # packed bytes by (N, K, group size, fp32 scales): a pure function of these


def _blob(packed, N: int, K: int, group_size: int, f32s: bool, index: int):
    key = (N, K, group_size, f32s)
    need = _blob_bytes.get(key)
    if need is None:
        lib = library()
        need = (lib.q4gsw_packed_bytes_f32s if f32s else lib.q4gsw_packed_bytes)(N, K, group_size)
        if len(_blob_bytes) < 4096:
            _blob_bytes[key] = need
    if not isinstance(packed, torch.Tensor) or packed.dtype is not _u8:
        raise TypeError("packed must be a uint8 tensor")
    if packed.get_device() != index or not packed.is_contiguous():
        raise ValueError(f"packed must be contiguous and on cuda:{index}")
    if packed.numel() < need:   # a shape that is not accepted needs 0: the call itself reports it
        raise ValueError(f"packed holds {packed.numel()} bytes, [{N}, {K}] at group size {group_size} needs {need}")
    return packed.data_ptr()


def _act(act: str, allowed=ACTS) -> int:
    code = allowed.get(act)
    if code is None:
        raise ValueError(f"act must be one of {tuple(allowed)} (got {act!r})")
    return code


_functions = {}


def _call(name: str, index: int, *args):
    """Call the C function with the device's current stream appended."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(library(), name)
    if index == _device_now():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(name, st)


def _out(t, name: str, dtype, shape, index: int):
    """(tensor, pointer) of an output: the caller's buffer, or a new one."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=index)
        return t, t.data_ptr()
    return t, _need(t, name, dtype, shape, index)


def q4gsw_prepack_gated(codes_gate, scales_gate, codes_up, scales_up, group_size: int, packed=None):
    """Gate and up projection (codes uint8 [F, K], scales fp16 or fp32 [K/gs, F] each) -> one packed blob
    of 2 F rows, row 2 j = gate row j, 2 j + 1 = up row j; fp32 scales give a layout-version-2 blob."""
    if not isinstance(codes_gate, torch.Tensor) or codes_gate.dim() != 2:
        raise ValueError("codes_gate must be a uint8 tensor of 2 dims")
    F, K = codes_gate.shape
    cg, _, index = _rows(codes_gate, "codes_gate", _u8, K)
    f32s = isinstance(scales_gate, torch.Tensor) and scales_gate.dtype == _f32
    sdt = _f32 if f32s else _f16
    sshape = (K // group_size if group_size > 0 else 0, F)
    sg = _need(scales_gate, "scales_gate", sdt, sshape, index)
    cu = _need(codes_up, "codes_up", _u8, (F, K), index)
    su = _need(scales_up, "scales_up", sdt, sshape, index)
    lib = library()
    nbytes = int((lib.q4gsw_packed_bytes_f32s if f32s else lib.q4gsw_packed_bytes)(2 * F, K, group_size))
    if packed is None:
        packed = _empty(max(nbytes, 1), dtype=_u8, device=index)
    elif not isinstance(packed, torch.Tensor):
        raise TypeError("packed must be a torch.Tensor")
    _call("q4gsw_prepack_gated_f32s" if f32s else "q4gsw_prepack_gated", index, cg, sg, cu, su, F, K, group_size,
          _need(packed, "packed", _u8, (packed.numel(),), index), packed.numel())
    return packed


def q4gsw_gated_fwd(packed, F: int, K: int, group_size: int, x, act: str = "silu", h=None, gu=None,
                    save_gu: bool = False, f32s: bool = False):
    """h = act(x Wg^T) * (x Wu^T): x fp16 [M, K] -> h fp16 [M, F].  With save_gu (or a gu buffer) returns
    (h, gu), gu fp16 [M, 2 F] the pairs the backward pass reads."""
    code = _act(act, _GATED)
    px, M, index = _rows(x, "x", _f16, K)
    pw = _blob(packed, 2 * F, K, group_size, f32s, index)
    h, ph = _out(h, "h", _f16, (M, F), index)
    pg = None
    if save_gu or gu is not None:
        gu, pg = _out(gu, "gu", _f16, (M, 2 * F), index)
    _call("q4gsw_gated_fwd_f32s" if f32s else "q4gsw_gated_fwd", index, pw, F, K, group_size, px, M, code, ph, pg)
    return h if gu is None else (h, gu)


def q4gsw_gated_bwd(packed, F: int, K: int, group_size: int, gu, d_h, act: str = "silu", d_gu=None, d_x=None,
                    f32s: bool = False):
    """(d_x fp16 [M, K], d_gu fp16 [M, 2 F]) from gu as saved by the forward and d_h fp16 [M, F].  d_gu may
    be gu's own buffer."""
    code = _act(act, _GATED)
    pd, M, index = _rows(d_h, "d_h", _f16, F)
    pg = _need(gu, "gu", _f16, (M, 2 * F), index)
    pw = _blob(packed, 2 * F, K, group_size, f32s, index)
    d_gu, pdg = _out(d_gu, "d_gu", _f16, (M, 2 * F), index)
    d_x, pdx = _out(d_x, "d_x", _f16, (M, K), index)
    _call("q4gsw_gated_bwd_f32s" if f32s else "q4gsw_gated_bwd", index, pw, F, K, group_size, pg, pd, M, code, pdg, pdx)
    return d_x, d_gu


def q4gsw_linear_act_fwd(packed, N: int, K: int, group_size: int, x, bias=None, act: str = "none", residual=None,
                         y=None, z=None, save_z: bool = False, f32s: bool = False):
    """y = act(x W^T + bias) + residual: x fp16 [M, K], bias fp16 [N], residual fp16 [M, N] -> y fp16 [M, N]
    (y may be the residual's buffer).  With save_z (or a z buffer) returns (y, z), z = x W^T + bias."""
    code = _act(act)
    px, M, index = _rows(x, "x", _f16, K)
    pw = _blob(packed, N, K, group_size, f32s, index)
    pb = None if bias is None else _need(bias, "bias", _f16, (N,), index)
    pr = None if residual is None else _need(residual, "residual", _f16, (M, N), index)
    y, py = _out(y, "y", _f16, (M, N), index)
    pz = None
    if save_z or z is not None:
        z, pz = _out(z, "z", _f16, (M, N), index)
    _call("q4gsw_linear_act_fwd_f32s" if f32s else "q4gsw_linear_act_fwd", index, pw, N, K, group_size, px, M, pb, code,
          pr, py, pz)
    return y if z is None else (y, z)


def q4gsw_linear_act_bwd(packed, N: int, K: int, group_size: int, d_y, z=None, act: str = "none", d_z=None, d_x=None,
                         d_bias=None, want_bias: bool = False, f32s: bool = False):
    """(d_x fp16 [M, K], d_z fp16 [M, N], d_bias fp32 [N]) from d_y fp16 [M, N] and, with an activation, z as
    saved by the forward.  d_z is None without an activation (it is d_y then), d_bias unless asked for (a buffer
    for it is 16-byte aligned, like every other)."""
    code = _act(act)
    pd, M, index = _rows(d_y, "d_y", _f16, N)
    pw = _blob(packed, N, K, group_size, f32s, index)
    pz = pdz = pb = None
    if code:
        if z is None:
            raise ValueError("z is required with an activation")
        pz = _need(z, "z", _f16, (M, N), index)
        d_z, pdz = _out(d_z, "d_z", _f16, (M, N), index)
    elif z is not None or d_z is not None:
        raise ValueError("without an activation there is no z and d_z is d_y")
    d_x, pdx = _out(d_x, "d_x", _f16, (M, K), index)
    if want_bias or d_bias is not None:
        d_bias, pb = _out(d_bias, "d_bias", _f32, (N,), index)
    _call("q4gsw_linear_act_bwd_f32s" if f32s else "q4gsw_linear_act_bwd", index, pw, N, K, group_size, pz, pd, M, code,
          pdz, pdx, pb)
    return d_x, d_z, d_bias


def _teacher(logits, indices, teacher):
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_f32, _f16):
        raise TypeError("logits must be a float32 or float16 tensor")
    if logits.dim() != 2:
        raise ValueError(f"logits must have 2 dims (got {logits.dim()})")
    if not isinstance(indices, torch.Tensor) or indices.dim() != 2:
        raise ValueError("indices must be an int32 tensor of 2 dims")
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in (_f32, _f16):
        raise TypeError("teacher must be a float32 or float16 tensor")
    V, k = logits.shape[1], indices.shape[1]
    pz, M, index = _rows(logits, "logits", logits.dtype, V)
    head = (pz, int(logits.dtype is _f16), M, V)
    tail = (_need(indices, "indices", _i32, (M, k), index), _need(teacher, "teacher", teacher.dtype, (M, k), index),
            int(teacher.dtype is _f16), k)
    return index, M, V, head, tail


def q4gsw_distill_fwd(logits, indices, teacher, temperature: float = 1.0, loss=None, lse=None):
    """(loss fp32 [M], lse fp32 [M]) of the student's logits [M, V] against the teacher's top logits [M, k] at
    token ids `indices` (int32, -1 = padding); fp32 or fp16 logits on either side."""
    index, M, V, head, tail = _teacher(logits, indices, teacher)
    loss, pl = _out(loss, "loss", _f32, (M,), index)
    lse, pe = _out(lse, "lse", _f32, (M,), index)
    _call("q4gsw_distill_fwd", index, *head, *tail, temperature, pl, pe)
    return loss, lse


def q4gsw_distill_bwd(logits, lse, indices, teacher, d_loss, temperature: float = 1.0, d_logits=None):
    """d_logits fp16 [M, V] from the forward's lse and d_loss fp32 [M], the gradient of each row's loss."""
    index, M, V, head, tail = _teacher(logits, indices, teacher)
    pe = _need(lse, "lse", _f32, (M,), index)
    pd = _need(d_loss, "d_loss", _f32, (M,), index)
    d_logits, pg = _out(d_logits, "d_logits", _f16, (M, V), index)
    _call("q4gsw_distill_bwd", index, *head, pe, *tail, temperature, pd, pg)
    return d_logits


def q4gsw_distill_step(logits, indices, teacher, d_loss, temperature: float = 1.0, loss=None, lse=None, d_logits=None):
    """(loss, lse, d_logits) in one pass over the logits, for a d_loss known beforehand."""
    index, M, V, head, tail = _teacher(logits, indices, teacher)
    pd = _need(d_loss, "d_loss", _f32, (M,), index)
    loss, pl = _out(loss, "loss", _f32, (M,), index)
    lse, pe = _out(lse, "lse", _f32, (M,), index)
    d_logits, pg = _out(d_logits, "d_logits", _f16, (M, V), index)
    _call("q4gsw_distill_step", index, *head, *tail, temperature, pd, pl, pe, pg)
    return loss, lse, d_logits
