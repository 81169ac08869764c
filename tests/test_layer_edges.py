"""Layer operators at the edges of their arguments: scales, values and sizes
far from the usual ones."""
import numpy as np
import pytest
import torch

import layers_ref as R
import test_layers as L

TYPES = L.TYPES


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,layout", [(8, "dense"), (33, "odd"), (250, "slice"), (1024, "dense"), (2049, "odd")])
@pytest.mark.parametrize("scale", [-1.5, float("inf"), float("-inf"), float("nan"), 0.0, -0.0])
def test_padding_is_zero_whatever_the_scale(v, dtype, d, layout, scale):
    g = L.gen(d)
    table = L.matrix(g, 40, d, dtype, layout)
    tokens = torch.tensor([3, -1, 39, 40, 0, 2 ** 40, 7], device="cuda")
    out = v.embedding(tokens, table, scale=scale, out=L.like(torch.empty(7, d, dtype=dtype, device="cuda"), layout))
    inside = [0, 2, 4, 6]
    want = (table[tokens[inside]].float() * scale).to(dtype)
    assert torch.equal(torch.nan_to_num(out[inside], 7.0), torch.nan_to_num(want, 7.0))
    bits = out[[1, 3, 5]].contiguous().view(torch.int32 if dtype == torch.float32 else torch.int16)
    assert not bits.any()  # +0
