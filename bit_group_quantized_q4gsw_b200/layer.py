"""The operators of include/q4gsw_layer.h on torch tensors: the gated
feed-forward block, the projection with an epilogue and the distillation loss.

Argument marshalling only, as in binding.py.  Besides dtype, contiguity and
device every shape is checked here, since the C calls see pointers alone.  The
calls run on the current stream of the tensors' device, whichever device is
current.
"""
from __future__ import annotations

import torch

from .binding import _check, library

ACTS = {"none": 0, "silu": 1, "gelu_tanh": 2}

# the current stream's handle without building a Stream object (2 us of a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # None in a build without CUDA

_f16, _f32, _i32, _u8 = torch.float16, torch.float32, torch.int32, torch.uint8


def _need(t, name: str, dtype, shape, device):
    """Check one tensor and return its pointer."""
    try:   # one test of everything: a call of a few microseconds spends as long on its arguments
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    raise ValueError(f"{name} must be contiguous")


def _first(t, name: str, dtype, ndim: int):
    """Check the tensor that fixes the device; returns its device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {t.dim()})")
    return t.device


def _blob(packed, N: int, K: int, group_size: int, f32s: bool, device):
    if not isinstance(packed, torch.Tensor) or packed.dtype != _u8:
        raise TypeError("packed must be a uint8 tensor")
    if packed.device != device or not packed.is_contiguous():
        raise ValueError(f"packed must be contiguous and on {device}")
    lib = _lib or _load()
    need = (lib.q4gsw_packed_bytes_f32s if f32s else lib.q4gsw_packed_bytes)(N, K, group_size)
    if packed.numel() < need:   # a shape that is not accepted needs 0: the call itself reports it
        raise ValueError(f"packed holds {packed.numel()} bytes, [{N}, {K}] at group size {group_size} needs {need}")
    return packed.data_ptr()


def _act(act: str, allowed=("none", "silu", "gelu_tanh")) -> int:
    if act not in allowed:
        raise ValueError(f"act must be one of {allowed} (got {act!r})")
    return ACTS[act]


_lib = None


def _load():
    global _lib
    _lib = library()
    return _lib


def _call(name: str, device, *args):
    """Call the C function with the device's current stream appended."""
    fn = getattr(_lib or _load(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(name, st)


def q4gsw_prepack_gated(codes_gate, scales_gate, codes_up, scales_up, group_size: int, packed=None):
    """Gate and up projection (codes uint8 [F, K], scales fp16 or fp32 [K/gs, F] each) -> one packed blob
    of 2 F rows, row 2 j = gate row j, 2 j + 1 = up row j; fp32 scales give a layout-version-2 blob."""
    dev = _first(codes_gate, "codes_gate", _u8, 2)
    F, K = codes_gate.shape
    f32s = isinstance(scales_gate, torch.Tensor) and scales_gate.dtype == _f32
    sdt = _f32 if f32s else _f16
    lib = _lib or _load()
    nbytes = int((lib.q4gsw_packed_bytes_f32s if f32s else lib.q4gsw_packed_bytes)(2 * F, K, group_size))
    if packed is None:
        packed = torch.empty(max(nbytes, 1), dtype=_u8, device=dev)
    sshape = (K // group_size if group_size > 0 else 0, F)
    _call("q4gsw_prepack_gated_f32s" if f32s else "q4gsw_prepack_gated", dev,
          _need(codes_gate, "codes_gate", _u8, (F, K), dev), _need(scales_gate, "scales_gate", sdt, sshape, dev), _need(codes_up, "codes_up", _u8, (F, K), dev),
          _need(scales_up, "scales_up", sdt, sshape, dev), F, K, group_size,
          _need(packed, "packed", _u8, (packed.numel(),), dev), packed.numel())
    return packed


def q4gsw_gated_fwd(packed, F: int, K: int, group_size: int, x, act: str = "silu", h=None, gu=None,
                    save_gu: bool = False, f32s: bool = False):
    """h = act(x Wg^T) * (x Wu^T): x fp16 [M, K] -> h fp16 [M, F].  With save_gu (or a gu buffer) returns
    (h, gu), gu fp16 [M, 2 F] the pairs the backward pass reads."""
    dev = _first(x, "x", _f16, 2)
    M = x.shape[0]
    if h is None:
        h = torch.empty((M, F), dtype=_f16, device=dev)
    if gu is None and save_gu:
        gu = torch.empty((M, 2 * F), dtype=_f16, device=dev)
    _call("q4gsw_gated_fwd_f32s" if f32s else "q4gsw_gated_fwd", dev, _blob(packed, 2 * F, K, group_size, f32s, dev),
          F, K, group_size, _need(x, "x", _f16, (M, K), dev), M, _act(act, ("silu", "gelu_tanh")),
          _need(h, "h", _f16, (M, F), dev), None if gu is None else _need(gu, "gu", _f16, (M, 2 * F), dev))
    return h if gu is None else (h, gu)


def q4gsw_gated_bwd(packed, F: int, K: int, group_size: int, gu, d_h, act: str = "silu", d_gu=None, d_x=None,
                    f32s: bool = False):
    """(d_x fp16 [M, K], d_gu fp16 [M, 2 F]) from gu as saved by the forward and d_h fp16 [M, F].  d_gu may
    be gu's own buffer."""
    dev = _first(d_h, "d_h", _f16, 2)
    M = d_h.shape[0]
    if d_gu is None:
        d_gu = torch.empty((M, 2 * F), dtype=_f16, device=dev)
    if d_x is None:
        d_x = torch.empty((M, K), dtype=_f16, device=dev)
    _call("q4gsw_gated_bwd_f32s" if f32s else "q4gsw_gated_bwd", dev, _blob(packed, 2 * F, K, group_size, f32s, dev),
          F, K, group_size, _need(gu, "gu", _f16, (M, 2 * F), dev), _need(d_h, "d_h", _f16, (M, F), dev), M,
          _act(act, ("silu", "gelu_tanh")), _need(d_gu, "d_gu", _f16, (M, 2 * F), dev),
          _need(d_x, "d_x", _f16, (M, K), dev))
    return d_x, d_gu


def q4gsw_linear_act_fwd(packed, N: int, K: int, group_size: int, x, bias=None, act: str = "none", residual=None,
                         y=None, z=None, save_z: bool = False, f32s: bool = False):
    """y = act(x W^T + bias) + residual: x fp16 [M, K], bias fp16 [N], residual fp16 [M, N] -> y fp16 [M, N]
    (y may be the residual's buffer).  With save_z (or a z buffer) returns (y, z), z = x W^T + bias."""
    dev = _first(x, "x", _f16, 2)
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=_f16, device=dev)
    if z is None and save_z:
        z = torch.empty((M, N), dtype=_f16, device=dev)
    _call("q4gsw_linear_act_fwd_f32s" if f32s else "q4gsw_linear_act_fwd", dev,
          _blob(packed, N, K, group_size, f32s, dev), N, K, group_size, _need(x, "x", _f16, (M, K), dev), M,
          None if bias is None else _need(bias, "bias", _f16, (N,), dev), _act(act),
          None if residual is None else _need(residual, "residual", _f16, (M, N), dev),
          _need(y, "y", _f16, (M, N), dev), None if z is None else _need(z, "z", _f16, (M, N), dev))
    return y if z is None else (y, z)


def q4gsw_linear_act_bwd(packed, N: int, K: int, group_size: int, d_y, z=None, act: str = "none", d_z=None, d_x=None,
                         d_bias=None, want_bias: bool = False, f32s: bool = False):
    """(d_x fp16 [M, K], d_z fp16 [M, N], d_bias fp32 [N]) from d_y fp16 [M, N] and, with an activation, z as
    saved by the forward.  d_z is None without an activation (it is d_y then), d_bias unless asked for."""
    dev = _first(d_y, "d_y", _f16, 2)
    M = d_y.shape[0]
    a = _act(act)
    if a and z is None:
        raise ValueError("z is required with an activation")
    if not a and (z is not None or d_z is not None):
        raise ValueError("without an activation there is no z and d_z is d_y")
    if a and d_z is None:
        d_z = torch.empty((M, N), dtype=_f16, device=dev)
    if d_x is None:
        d_x = torch.empty((M, K), dtype=_f16, device=dev)
    if d_bias is None and want_bias:
        d_bias = torch.empty((N,), dtype=_f32, device=dev)
    _call("q4gsw_linear_act_bwd_f32s" if f32s else "q4gsw_linear_act_bwd", dev,
          _blob(packed, N, K, group_size, f32s, dev), N, K, group_size,
          _need(z, "z", _f16, (M, N), dev) if a else None, _need(d_y, "d_y", _f16, (M, N), dev), M, a,
          _need(d_z, "d_z", _f16, (M, N), dev) if a else None, _need(d_x, "d_x", _f16, (M, K), dev),
          None if d_bias is None else _need(d_bias, "d_bias", _f32, (N,), dev))
    return d_x, d_z, d_bias


def _teacher(logits, indices, teacher):
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_f32, _f16):
        raise TypeError("logits must be a float32 or float16 tensor")
    dev = _first(logits, "logits", logits.dtype, 2)
    if not isinstance(indices, torch.Tensor) or indices.dim() != 2:
        raise ValueError("indices must be an int32 tensor of 2 dims")
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in (_f32, _f16):
        raise TypeError("teacher must be a float32 or float16 tensor")
    M, V = logits.shape
    k = indices.shape[1]
    head = (_need(logits, "logits", logits.dtype, (M, V), dev), int(logits.dtype == _f16), M, V)
    tail = (_need(indices, "indices", _i32, (M, k), dev), _need(teacher, "teacher", teacher.dtype, (M, k), dev),
            int(teacher.dtype == _f16), k)
    return dev, M, V, head, tail


def q4gsw_distill_fwd(logits, indices, teacher, temperature: float = 1.0, loss=None, lse=None):
    """(loss fp32 [M], lse fp32 [M]) of the student's logits [M, V] against the teacher's top logits [M, k] at
    token ids `indices` (int32, -1 = padding); fp32 or fp16 logits on either side."""
    dev, M, V, head, tail = _teacher(logits, indices, teacher)
    if loss is None:
        loss = torch.empty(M, dtype=_f32, device=dev)
    if lse is None:
        lse = torch.empty(M, dtype=_f32, device=dev)
    _call("q4gsw_distill_fwd", dev, *head, *tail, temperature, _need(loss, "loss", _f32, (M,), dev),
          _need(lse, "lse", _f32, (M,), dev))
    return loss, lse


def q4gsw_distill_bwd(logits, lse, indices, teacher, d_loss, temperature: float = 1.0, d_logits=None):
    """d_logits fp16 [M, V] from the forward's lse and d_loss fp32 [M], the gradient of each row's loss."""
    dev, M, V, head, tail = _teacher(logits, indices, teacher)
    if d_logits is None:
        d_logits = torch.empty((M, V), dtype=_f16, device=dev)
    _call("q4gsw_distill_bwd", dev, *head, _need(lse, "lse", _f32, (M,), dev), *tail, temperature,
          _need(d_loss, "d_loss", _f32, (M,), dev), _need(d_logits, "d_logits", _f16, (M, V), dev))
    return d_logits


def q4gsw_distill_step(logits, indices, teacher, d_loss, temperature: float = 1.0, loss=None, lse=None, d_logits=None):
    """(loss, lse, d_logits) in one pass over the logits, for a d_loss known beforehand."""
    dev, M, V, head, tail = _teacher(logits, indices, teacher)
    if loss is None:
        loss = torch.empty(M, dtype=_f32, device=dev)
    if lse is None:
        lse = torch.empty(M, dtype=_f32, device=dev)
    if d_logits is None:
        d_logits = torch.empty((M, V), dtype=_f16, device=dev)
    _call("q4gsw_distill_step", dev, *head, *tail, temperature, _need(d_loss, "d_loss", _f32, (M,), dev),
          _need(loss, "loss", _f32, (M,), dev), _need(lse, "lse", _f32, (M,), dev),
          _need(d_logits, "d_logits", _f16, (M, V), dev))
    return loss, lse, d_logits
