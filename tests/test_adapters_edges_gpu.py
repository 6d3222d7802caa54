"""Adapters of many requests at the edges of what a call allows: plans that are shorter than the call's."""
import numpy as np
import pytest
import torch

from helpers import cuda
from test_adapters_gpu import head, make, q

pytestmark = pytest.mark.gpu


def c_call(name, *args):
    """The C function on the current stream, with tensors as their addresses: no check of Python's before it."""
    from bit_group_quantized_q4gsw_b200 import binding as b
    at = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    return getattr(b.library(), name)(*at, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("M", [12, 100, 600, 4100])
def test_a_plan_that_ends_before_the_calls_is_not_read_past_its_head(M):
    # the C calls have no size of the plan: the plan of one token, in a buffer of its own size, for M tokens.  The other
    # parts of a plan of M tokens would lie behind that buffer.
    m = q()
    N, K, gs, L, r = 64, 128, 32, 3, 8
    c = make(M, N, K, gs, L, r, np.arange(M) % L)
    blob, _, _, _, _, a, b = head(c)
    short = m.q4gsw_adapters_plan(torch.zeros(1, dtype=torch.int32, device="cuda"), L)
    assert 4 * short.numel() == 4 * (4 + 8 + 4 + 4 + 16 + 4)      # head, first, order, one tile, its rows, a pair
    x, d_y = cuda(c["x"]), cuda(c["d_y"])
    y, u, v = torch.zeros(M, N, device="cuda").half(), torch.full((M, r), 7.0, device="cuda"), torch.full((M, r), 7.0, device="cuda")
    d_x, d_a, d_b = torch.zeros(M, K, device="cuda").half(), torch.full((L, r, K), 5.0, device="cuda"), torch.full((L, N, r), 5.0, device="cuda")
    m.q4gsw_device_error_check()
    assert c_call("q4gsw_adapters_fwd", blob, N, K, gs, short, a, b, None, L, r, x, M, None, None, y, u) == 0
    with pytest.raises(m.Q4gswError, match="INDEX"):
        m.q4gsw_device_error_check()
    assert (u == 7).all()
    assert c_call("q4gsw_adapters_bwd", blob, N, K, gs, short, a, b, None, L, r, x, u, d_y, M, 0, v, d_x, d_a, d_b) == 0
    with pytest.raises(m.Q4gswError, match="INDEX"):
        m.q4gsw_device_error_check()
    assert (v == 7).all() and (d_a == 5).all() and (d_b == 5).all()
    m.q4gsw_adapters_fwd(*head(c), x)                              # the right plan still serves
    m.q4gsw_device_error_check()
