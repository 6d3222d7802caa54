"""The clip of gradients whose factor or norm is outside fp32's normal numbers."""
import math

import numpy as np
import pytest
import torch

from oracle import q4gsw_adapters as oa
from test_grads_gpu import host, lists, q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [[3000, 17], [200000, 5, 70001]])      # one launch, two
@pytest.mark.parametrize("size,max_norm,inv", [(1e36, 1e-6, 1.0), (3e37, 1e-3, 1.0), (1e30, 1e-6, 1e-9), (1e-3, 1.0, 1e-43), (1e-30, 1e-38, 1.0),
                                               (1e25, 1e-30, 2.0 ** -16), (3e37, 1.0, -1.0)])
def test_factors_below_the_normal_numbers_keep_their_bits(sizes, size, max_norm, inv):
    # 1e36 clipped to 1e-6 over 5000 values: a factor of 1e-44 or so, of which fp32 holds three bits, and values of 1e-8
    m = q()
    g = lists(sizes, [0] * len(sizes), sigma=size)
    inv = float(np.float32(inv))
    before = [host(t) for t in g]
    max_norm = float(np.float32(max_norm))
    outs = [torch.zeros_like(t) for t in g]
    norm = m.q4gsw_grad_clip(m.q4gsw_grad_set(g, outs), max_norm, inv_scale=inv)
    n, b = oa.grad_norm(before, inv)
    assert math.isinf(norm.item()) if n > 3.5e38 else abs(norm.item() - n) <= b
    for out, (want, bound) in zip(outs, oa.grad_clip(before, max_norm, inv)):
        assert (np.abs(host(out).astype(np.float64) - want) <= bound).all()


def test_a_finite_list_whose_norm_is_beyond_fp32_is_clipped():
    m = q()
    for count in (4, 300000):
        g = [torch.full((count,), 3e38, device="cuda")]
        norm = m.q4gsw_grad_clip(m.q4gsw_grad_set(g), 2.0)
        assert math.isinf(norm.item())
        want = 2.0 / math.sqrt(count)
        assert ((g[0].double() - want).abs() <= 8 * 2.0 ** -24 * want).all()
