"""The layers around the attention on the GPU: waits, values, streams and sizes
at their ends, against float64 references (oracle/layers.py) within the error
bounds that test_layers_gpu.py derives."""

import math

import pytest

from test_layers_gpu import _check_cross, _cross_case, _run_cross

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ cross attention

@pytest.mark.parametrize("lq,lk", [([300], [6401]), ([40, 130], [3333, 4100]), ([1], [20001]),
                                   ([128] * 6, [1025, 1, 900, 2049, 127, 1300])])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(4, 4, 128, "bf16"), (8, 2, 64, "fp16")])
def test_cross_long_unmasked_segments_that_end_inside_a_tile(lq, lk, Hq, Hk, D, dtype):
    """Many value tiles that need nothing, then one whose last rows must not count:
    the warp that writes zeros there is at that tile and no other."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq + [0], lk + [200], Hq, Hk, D, dtype)
    cu_q, cu_k = cu_q[:-1].contiguous(), cu_k[:-1].contiguous()
    n = sum(lk)
    k[n:], v[n:] = math.nan, math.inf
    first = None
    for _ in range(10):
        o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
        if first is None:
            first = o
            _check_cross(q, k[:n], v[:n], cu_q, cu_k, o, lse, D ** -0.5, None, "o")
        assert torch.equal(o, first)
