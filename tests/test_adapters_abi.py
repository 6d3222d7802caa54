"""Host-side checks of include/q4gsw_adapters.h: every declared function is
exported and bound, and bad arguments are refused before the device is touched."""
import ctypes
import os
import re

import pytest
import torch

import bit_group_quantized_q4gsw_b200 as q
from bit_group_quantized_q4gsw_b200 import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000   # an aligned address that is never dereferenced
OK, NULL, SHAPE, ALIGN, UNSUPPORTED, SIZE = 0, 1, 2, 3, 4, 7
BIG = 1 << 40


def test_header_library_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "q4gsw_adapters.h")).read()
    names = re.findall(r"Q4GSW_API\s+[\w\s\*]*?\b(q4gsw_\w+)\s*\(", text)
    assert sorted(names) == sorted(n for n, _, _ in b.ADAPTER_SIGNATURES)
    for n in names:
        assert hasattr(b.library(), n), n


def test_plan_arguments_and_size():
    lib = b.library()
    for M, L in ((-1, 4), (4, 0), (4, 1025), ((1 << 27) + 1, 4)):
        assert lib.q4gsw_adapters_plan_bytes(M, L) == 0
        assert lib.q4gsw_adapters_plan(P, M, L, P, BIG, None) == SHAPE
    need = lib.q4gsw_adapters_plan_bytes(100, 7)
    # head 4, first 9 -> 12, order 100, (100 + 15 * 8) / 16 = 13 -> 16 tiles, 13 * 16 rows, (13 + 8) / 2 = 10 -> 12 pairs
    assert need == 4 * (4 + 12 + 100 + 16 + 13 * 16 + 12)
    assert lib.q4gsw_adapters_plan(P, 100, 7, P, need - 1, None) == SIZE
    assert lib.q4gsw_adapters_plan(None, 100, 7, P, need, None) == NULL
    assert lib.q4gsw_adapters_plan(P, 100, 7, None, need, None) == NULL
    assert lib.q4gsw_adapters_plan(P + 2, 100, 7, P, need, None) == ALIGN
    assert lib.q4gsw_adapters_plan(P, 100, 7, P + 4, need, None) == ALIGN
    assert lib.q4gsw_adapters_plan(None, 0, 7, None, 0, None) == OK


@pytest.mark.parametrize("suffix", ["", "_f32s"])
def test_adapters_arguments(suffix):
    lib = b.library()
    f, g = getattr(lib, "q4gsw_adapters_fwd" + suffix), getattr(lib, "q4gsw_adapters_bwd" + suffix)

    def fwd(N=64, K=128, gs=32, L=3, r=16, M=4, packed=P, plan=P, a=P, bb=P, scale=None, x=P, bias=None, res=None, y=P, u=P):
        return f(packed, N, K, gs, plan, a, bb, scale, L, r, x, M, bias, res, y, u, None)

    def bwd(N=64, K=128, gs=32, L=3, r=16, M=4, packed=P, plan=P, a=P, bb=P, scale=None, x=P, u=P, d_y=P, acc=0, v=P, d_x=P,
            d_a=P, d_b=P):
        return g(packed, N, K, gs, plan, a, bb, scale, L, r, x, u, d_y, M, acc, v, d_x, d_a, d_b, None)

    for kw, st in ((dict(N=0), SHAPE), (dict(N=62), SHAPE), (dict(N=68), ALIGN), (dict(K=96), ALIGN),
                   (dict(gs=48), UNSUPPORTED), (dict(L=0), SHAPE), (dict(L=1025), SHAPE), (dict(r=0), SHAPE),
                   (dict(r=12), SHAPE), (dict(r=72), SHAPE), (dict(M=-1), SHAPE), (dict(M=1 << 28), SHAPE),
                   (dict(N=64 * 65536), SHAPE), (dict(K=64 * 65536), SHAPE), (dict(packed=None), NULL),
                   (dict(plan=None), NULL), (dict(a=None), NULL), (dict(bb=None), NULL), (dict(x=None), NULL),
                   (dict(u=None), NULL), (dict(packed=P + 8), ALIGN), (dict(plan=P + 4), ALIGN), (dict(a=P + 2), ALIGN),
                   (dict(bb=P + 8), ALIGN), (dict(scale=P + 2), ALIGN), (dict(x=P + 8), ALIGN), (dict(u=P + 4), ALIGN)):
        assert (fwd(**kw), bwd(**kw)) == (st, st), kw
    for kw, st in ((dict(y=None), NULL), (dict(y=P + 8), ALIGN), (dict(bias=P + 2), ALIGN), (dict(res=P + 8), ALIGN)):
        assert fwd(**kw) == st, kw
    for kw, st in ((dict(d_y=None), NULL), (dict(v=None), NULL), (dict(d_a=None), NULL), (dict(d_b=None), NULL),
                   (dict(d_x=None, d_a=None, d_b=None), NULL), (dict(d_y=P + 8), ALIGN), (dict(v=P + 4), ALIGN),
                   (dict(d_x=P + 8), ALIGN), (dict(d_a=P + 4), ALIGN), (dict(d_b=P + 8), ALIGN)):
        assert bwd(**kw) == st, kw
    assert fwd(M=0, packed=None, plan=None, a=None, bb=None, x=None, y=None, u=None) == OK
    assert b.q4gsw_last_route() == "empty"
    assert bwd(M=0, acc=1, packed=None, plan=None, a=None, bb=None, x=None, u=None, d_y=None, v=None) == OK


@pytest.mark.parametrize("suffix", ["", "_f32s"])
def test_outputs_in_the_place_of_what_is_read_behind_them_are_refused(suffix):
    lib = b.library()
    f, g = getattr(lib, "q4gsw_adapters_fwd" + suffix), getattr(lib, "q4gsw_adapters_bwd" + suffix)
    q = P + 4096
    assert f(P, 64, 64, 32, P, P, P, None, 3, 16, q, 4, None, q, q, P, None) == UNSUPPORTED      # y = x = the residual
    for x, u, d_y, v, d_x, d_a in ((P, P, q, q, q, P), (P, P, q, q, q, None), (q, P, P, q, q, P), (P, q, P, q, None, P)):
        assert g(P, 64, 64, 32, P, P, P, None, 3, 16, x, u, d_y, 4, 0, v, d_x, d_a, d_a, None) == UNSUPPORTED


def test_norms_arguments():
    lib = b.library()

    def fwd(M=4, D=64, h=P, block=P, post=P, gate=P, rows=0, f=1.0, pre=P, o=0.0, eps=1e-6, out=P, x=P):
        return lib.q4gsw_norms_fwd(h, block, post, gate, rows, f, pre, o, eps, M, D, out, x, None)

    def bwd(M=4, D=64, h=P, dx=P, dh=P, block=P, post=P, gate=P, rows=0, f=1.0, pre=P, o=0.0, eps=1e-6, dr=P, db=P, dgr=None,
            dpre=P, dpost=P, dg=P, ws=P, n=BIG):
        return lib.q4gsw_norms_bwd(h, dx, dh, block, post, gate, rows, f, pre, o, eps, M, D, dr, db, dgr, dpre, dpost, dg, ws,
                                   n, None)

    inf, nan = float("inf"), float("nan")
    for kw, st in ((dict(M=-1), SHAPE), (dict(M=(1 << 30) + 1), SHAPE), (dict(D=0), SHAPE), (dict(D=62), SHAPE), (dict(D=60), ALIGN), (dict(D=32776), SHAPE),
                   (dict(f=inf), SHAPE), (dict(o=nan), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=nan), SHAPE),
                   (dict(rows=2), UNSUPPORTED), (dict(h=None), NULL), (dict(block=None), NULL), (dict(pre=None), NULL),
                   (dict(h=P + 8), ALIGN), (dict(block=P + 8), ALIGN), (dict(post=P + 2), ALIGN), (dict(gate=P + 2), ALIGN),
                   (dict(pre=P + 8), ALIGN)):
        assert (fwd(**kw), bwd(**kw)) == (st, st), kw
    for kw, st in ((dict(x=None), NULL), (dict(x=None, pre=None, out=None), NULL), (dict(out=P + 8), ALIGN), (dict(x=P + 8), ALIGN)):
        assert fwd(**kw) == st, kw
    for kw, st in ((dict(dx=None), NULL), (dict(dx=None, dh=None, pre=None, dpre=None), NULL), (dict(dr=None), NULL),
                   (dict(db=None), NULL), (dict(dgr=P), NULL), (dict(rows=1), NULL), (dict(rows=1, dgr=P), NULL),
                   (dict(post=None), NULL), (dict(gate=None), NULL), (dict(ws=None), NULL), (dict(dx=P + 8), ALIGN),
                   (dict(dh=P + 8), ALIGN), (dict(dr=P + 8), ALIGN), (dict(db=P + 8), ALIGN), (dict(dpre=P + 4), ALIGN),
                   (dict(dg=P + 4), ALIGN), (dict(ws=P + 4), ALIGN), (dict(rows=1, dgr=P + 8, dg=None), ALIGN)):
        assert bwd(**kw) == st, kw
    need = lib.q4gsw_norms_workspace_bytes(4, 64)
    assert need > 0 and bwd(n=need - 1) == SIZE
    assert lib.q4gsw_norms_workspace_bytes(4, 60) == 0
    assert fwd(M=0, h=None, out=None, x=None) == OK
    assert bwd(M=0, h=None, dpre=None, dpost=None, dg=None) == OK


def _table(lib, sizes, grads=None, hg=None, outs="same", ho=None, nbytes=None, count=None):
    n = len(sizes)
    arr = lambda t, v: None if v is None else (t * n)(*v)      # noqa: E731
    grads = [P] * n if grads is None else grads
    outs = grads if outs == "same" else outs
    hg = [0] * n if hg is None else hg
    ho = hg if ho is None else ho
    s = arr(ctypes.c_int64, sizes)
    need = lib.q4gsw_grad_table_bytes(n, s)
    host = ctypes.create_string_buffer(max(int(need), 1))
    st = lib.q4gsw_grad_table(n if count is None else count, arr(ctypes.c_void_p, grads), arr(ctypes.c_int, hg),
                              arr(ctypes.c_void_p, outs), None if outs is None else arr(ctypes.c_int, ho), s, host,
                              need if nbytes is None else nbytes)
    return st, need


def test_grad_table_arguments():
    lib = b.library()
    assert _table(lib, [5, 0, 8193])[0] == OK
    assert _table(lib, [5, 0, 8193])[1] == 32 * (1 + 0 + 9)        # a record of 32 bytes for every 1024 elements
    assert _table(lib, [5], outs=None)[0] == OK
    assert _table(lib, [5, 0], grads=[P, None])[0] == OK           # an empty tensor has no address
    for kw, st in ((dict(count=0), SHAPE), (dict(count=65537), SHAPE), (dict(hg=[2]), UNSUPPORTED), (dict(hg=[0], ho=[3]), UNSUPPORTED),
                   (dict(grads=[None]), NULL), (dict(outs=[None]), NULL), (dict(grads=[P + 2]), ALIGN),
                   (dict(grads=[P + 1], hg=[1]), ALIGN), (dict(outs=[P + 2]), ALIGN), (dict(nbytes=31), SIZE)):
        assert _table(lib, [5], **kw)[0] == st, kw
    assert _table(lib, [5], grads=[P + 2], hg=[1])[0] == OK
    assert _table(lib, [-1], nbytes=1)[0] == SHAPE
    assert _table(lib, [1 << 45]) == (SIZE, 0)
    assert _table(lib, [1024 << 26])[1] == 0
    assert lib.q4gsw_grad_table_bytes(0, None) == 0


def test_grad_call_arguments():
    lib = b.library()
    w = lib.q4gsw_grad_workspace_bytes()
    for kw, st in ((dict(inv=float("nan")), SHAPE), (dict(inv=float("inf")), SHAPE),
                   (dict(table=None), NULL), (dict(norm=None), NULL), (dict(ws=None), NULL), (dict(table=P + 8), ALIGN),
                   (dict(norm=P + 2), ALIGN), (dict(ws=P + 8), ALIGN), (dict(tb=16), SIZE), (dict(tb=48), SIZE),
                   (dict(tb=0), SIZE), (dict(tb=32 << 31), SIZE), (dict(wb=w - 1), SIZE)):
        a = dict(table=P, tb=1 << 20, inv=1.0, norm=P, ws=P, wb=w)
        a.update(kw)
        tail = (a["norm"], a["ws"], a["wb"], None)
        assert lib.q4gsw_grad_norm(a["table"], a["tb"], a["inv"], *tail) == st, kw
        assert lib.q4gsw_grad_clip(a["table"], a["tb"], 1.0, a["inv"], *tail) == st, kw
    # up to 64 records no workspace is looked at; one more needs it (and its size)
    assert lib.q4gsw_grad_norm(P, 65 * 32, 1.0, P, None, 0, None) == NULL
    assert lib.q4gsw_grad_clip(P, 65 * 32, 1.0, 1.0, P, P, 0, None) == SIZE
    assert lib.q4gsw_grad_norm(P, 64 * 32, 1.0, P, P + 8, 0, None) == ALIGN
    for m in (0.0, -1.0, float("nan")):
        assert lib.q4gsw_grad_clip(P, 1 << 20, m, 1.0, P, P, w, None) == SHAPE


def test_python_entry_points_refuse_tensors_off_the_device():
    x = torch.zeros(2, 128, dtype=torch.float16)
    blob = torch.zeros(1 << 16, dtype=torch.uint8)
    a, bb = torch.zeros(3, 8, 128, dtype=torch.float16), torch.zeros(3, 64, 8, dtype=torch.float16)
    plan = torch.zeros(1 << 12, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_adapters_plan(torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_adapters_fwd(blob, 64, 128, 32, plan, a, bb, x)
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_adapters_bwd(blob, 64, 128, 32, plan, a, bb, x, torch.zeros(2, 8), torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_norms_fwd(x, w_pre=x[0])
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_norms_bwd(x, d_x=x, w_pre=x[0])
    with pytest.raises(ValueError, match="CUDA"):
        q.q4gsw_grad_set([torch.zeros(4)])
    with pytest.raises(ValueError, match="empty"):
        q.q4gsw_grad_set([])
    with pytest.raises(TypeError, match="GradSet"):
        q.q4gsw_grad_norm([torch.zeros(4)])
    with pytest.raises(ValueError, match="2 dims"):
        q.q4gsw_norms_fwd(x[0])
    with pytest.raises(ValueError, match="1 dim"):
        q.q4gsw_adapters_plan(torch.zeros(4, 2, dtype=torch.int32), 3)
