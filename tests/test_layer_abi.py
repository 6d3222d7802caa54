"""Host-side checks of include/q4gsw_layer.h: every declared function is
exported and bound, and bad arguments are refused before the device is touched."""
import os
import re

import pytest
import torch

import bit_group_quantized_q4gsw_b200 as q
from bit_group_quantized_q4gsw_b200 import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000   # an aligned address that is never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, SIZE = 1, 2, 3, 4, 7


def test_header_library_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "q4gsw_layer.h")).read()
    names = re.findall(r"Q4GSW_API\s+[\w\s\*]*?\b(q4gsw_\w+)\s*\(", text)
    assert sorted(names) == sorted(n for n, _, _ in b.LAYER_SIGNATURES)
    for n in names:
        assert hasattr(b.library(), n), n


@pytest.mark.parametrize("suffix", ["", "_f32s"])
def test_gated_arguments(suffix):
    lib = b.library()
    pre, fwd, bwd = (getattr(lib, n + suffix) for n in ("q4gsw_prepack_gated", "q4gsw_gated_fwd", "q4gsw_gated_bwd"))
    need = int(getattr(lib, "q4gsw_packed_bytes" + suffix)(128, 128, 32))
    assert pre(P, P, P, P, 64, 128, 32, P, need - 1, None) == SIZE
    for hole in range(4):
        a = [P, P, P, P]
        a[hole] = None
        assert pre(*a, 64, 128, 32, P, need, None) == NULL
        a[hole] = P + 8
        assert pre(*a, 64, 128, 32, P, need, None) == ALIGN
    for F, K, gs, st in ((0, 128, 32, SHAPE), (-8, 128, 32, SHAPE), (62, 128, 32, SHAPE), (60, 128, 32, ALIGN),
                         (64, 96, 32, ALIGN), (64, 130, 32, SHAPE), (64, 128, 48, UNSUPPORTED),
                         (64, 128, 256, UNSUPPORTED), (0x40000000, 128, 32, SHAPE)):
        assert pre(P, P, P, P, F, K, gs, P, 1 << 40, None) == st, (F, K, gs)
        assert fwd(P, F, K, gs, P, 4, 1, P, P, None) == st, (F, K, gs)
        assert bwd(P, F, K, gs, P, P, 4, 1, P, P, None) == st, (F, K, gs)
    assert fwd(P, 64, 128, 32, P, -1, 1, P, P, None) == SHAPE
    assert bwd(P, 64, 128, 32, P, P, -1, 1, P, P, None) == SHAPE
    for act in (-1, 0, 3):
        assert fwd(P, 64, 128, 32, P, 4, act, P, P, None) == UNSUPPORTED
        assert bwd(P, 64, 128, 32, P, P, 4, act, P, P, None) == UNSUPPORTED
    assert fwd(None, 64, 128, 32, P, 4, 1, P, None, None) == NULL
    assert fwd(P, 64, 128, 32, None, 4, 1, P, None, None) == NULL
    assert fwd(P, 64, 128, 32, P, 4, 1, None, None, None) == NULL
    assert fwd(P, 64, 128, 32, P, 4, 1, P + 2, None, None) == ALIGN
    assert fwd(P, 64, 128, 32, P, 4, 1, P, P + 8, None) == ALIGN
    for hole in range(4):
        a = [P, P, P, P]
        a[hole] = None
        assert bwd(P, 64, 128, 32, a[0], a[1], 4, 1, a[2], a[3], None) == NULL
        a[hole] = P + 4
        assert bwd(P, 64, 128, 32, a[0], a[1], 4, 1, a[2], a[3], None) == ALIGN
    assert fwd(None, 64, 128, 32, None, 0, 1, None, None, None) == 0     # empty batch
    assert b.q4gsw_last_route() == "empty"
    assert bwd(None, 64, 128, 32, None, None, 0, 2, None, None, None) == 0


@pytest.mark.parametrize("suffix", ["", "_f32s"])
def test_linear_act_arguments(suffix):
    lib = b.library()
    fwd, bwd = (getattr(lib, n + suffix) for n in ("q4gsw_linear_act_fwd", "q4gsw_linear_act_bwd"))
    for N, K, gs, st in ((0, 128, 32, SHAPE), (62, 128, 32, SHAPE), (68, 128, 32, ALIGN), (64, 96, 32, ALIGN),
                         (64, 128, 8, UNSUPPORTED)):
        assert fwd(P, N, K, gs, P, 4, None, 0, None, P, None, None) == st
        assert bwd(P, N, K, gs, P, P, 4, 1, P, P, None, None) == st
    for act in (-1, 3):
        assert fwd(P, 64, 128, 32, P, 4, None, act, None, P, None, None) == UNSUPPORTED
        assert bwd(P, 64, 128, 32, P, P, 4, act, P, P, None, None) == UNSUPPORTED
    assert fwd(P, 64, 128, 32, P, -1, None, 0, None, P, None, None) == SHAPE
    assert fwd(P, 64, 128, 32, None, 4, None, 0, None, P, None, None) == NULL
    assert fwd(P, 64, 128, 32, P, 4, None, 0, None, None, None, None) == NULL
    for bias, res, y, z in ((P + 2, None, P, None), (None, P + 4, P, None), (None, None, P + 8, None),
                            (None, None, P, P + 2)):
        assert fwd(P, 64, 128, 32, P, 4, bias, 0, res, y, z, None) == ALIGN
    assert bwd(P, 64, 128, 32, None, P, 4, 1, P, P, None, None) == NULL      # z missing
    assert bwd(P, 64, 128, 32, P, P, 4, 1, None, P, None, None) == NULL      # d_z missing
    assert bwd(P, 64, 128, 32, None, None, 4, 0, None, P, None, None) == NULL
    assert bwd(P, 64, 128, 32, None, P, 4, 0, None, P + 8, None, None) == ALIGN
    assert bwd(P, 64, 128, 32, None, P, 4, 0, None, P, P + 4, None) == ALIGN
    assert fwd(None, 64, 128, 32, None, 0, None, 0, None, None, None, None) == 0
    assert bwd(None, 64, 128, 32, None, None, 0, 0, None, None, None, None) == 0


def test_distill_arguments():
    lib = b.library()

    def calls(M=4, V=64, k=4, T=1.0, hl=0, ht=0, z=P, i=P, t=P, lse=P, d=P, loss=P, g=P):
        return (lib.q4gsw_distill_fwd(z, hl, M, V, i, t, ht, k, T, loss, lse, None),
                lib.q4gsw_distill_bwd(z, hl, M, V, lse, i, t, ht, k, T, d, g, None),
                lib.q4gsw_distill_step(z, hl, M, V, i, t, ht, k, T, d, loss, lse, g, None))

    for kw, st in ((dict(M=-1), SHAPE), (dict(V=0), SHAPE), (dict(V=62), SHAPE), (dict(V=60), ALIGN),
                   (dict(k=0), SHAPE), (dict(k=1025), SHAPE), (dict(T=0.0), SHAPE), (dict(T=-1.0), SHAPE),
                   (dict(T=float("inf")), SHAPE), (dict(T=float("nan")), SHAPE), (dict(T=1e-39), SHAPE), (dict(T=1e19), SHAPE), (dict(hl=2), UNSUPPORTED),
                   (dict(ht=-1), UNSUPPORTED), (dict(M=0x7fffffff), SHAPE), (dict(z=None), NULL), (dict(i=None), NULL),
                   (dict(t=None), NULL), (dict(lse=None), NULL), (dict(z=P + 8), ALIGN), (dict(i=P + 2), ALIGN),
                   (dict(t=P + 2), ALIGN), (dict(t=P + 1, ht=1), ALIGN), (dict(lse=P + 2), ALIGN)):
        assert calls(**kw) == (st, st, st), kw
    f, bw, s = calls(loss=None)
    assert (f, s) == (NULL, NULL)
    assert calls(d=None)[1:] == (NULL, NULL) and calls(g=None)[1:] == (NULL, NULL)
    assert calls(d=P + 2)[1:] == (ALIGN, ALIGN) and calls(g=P + 8)[1:] == (ALIGN, ALIGN)
    assert calls(M=0, z=None, i=None, t=None, lse=None, d=None, loss=None, g=None) == (0, 0, 0)


def test_python_entry_points_refuse_tensors_off_the_device():
    x = torch.zeros(2, 128, dtype=torch.float16)
    blob = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_gated_fwd(blob, 64, 128, 32, x)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_linear_act_fwd(blob, 64, 128, 32, x)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_distill_fwd(torch.zeros(2, 64), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4))
    with pytest.raises(TypeError, match="float"):
        q.q4gsw_distill_fwd(torch.zeros(2, 64, dtype=torch.float64), torch.zeros(2, 4), torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_prepack_gated(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(4, 64, dtype=torch.float16),
                              torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(4, 64, dtype=torch.float16), 32)
