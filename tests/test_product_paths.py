"""The products' rarer ways through the tiles, each reached by sizes of its own:
sums that are both cut into splits and added up in chunks, sums longer than a
chunk of bf16 results, backward products in a launch each, one weight's gradient
alone; operands at the ends of their range.  Against the 64-bit definitions and
bounds of products_ref.py."""
import pytest
import torch

import products_ref as R
from test_layers import gen, matrix
from test_products import TYPES, near


@pytest.fixture(scope="module")
def v():
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    return vc


def splits_room(v, n, D, F, dtype):
    """Bytes of the workspace that the splits' sums of a gated block take."""
    if dtype == torch.bfloat16:
        return v.gated_ff_workspace_bytes(n, D, F, dtype, 1)
    wide = (D + 63) // 64 * 64 * 2 * 3  # a row laid out as three parts
    laid = sum((rows * wide + 255) // 256 * 256 for rows in (n, F, F))
    return v.gated_ff_workspace_bytes(n, D, F, dtype, 0) - laid


# Single CTAs and pairs whose tiles have 256 columns: two warps share a tile's rows,
# and a unit's sum is taken out of the tensor cores in several chunks.
SPLIT = [(torch.float32, 100, 1024, 4096), (torch.float32, 128, 4096, 4096), (torch.float32, 64, 2048, 4096),
         (torch.float32, 512, 4096, 2671), (torch.bfloat16, 700, 100000, 1000)]


def test_these_blocks_are_cut_into_splits(v):
    for dtype, n, D, F in SPLIT:
        rows = min(n, 128 if n <= 128 else 256)
        assert splits_room(v, n, D, F, dtype) >= 2 * rows * 256 * 4, (n, D, F)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,n,D,F", SPLIT)
def test_splits_of_a_gated_block_in_chunks(v, dtype, n, D, F):
    g = gen(n + D)
    x, wg, wu = matrix(g, n, D, dtype), matrix(g, F, D, dtype, scale=0.03), matrix(g, F, D, dtype, scale=0.03)
    if D > 4096:  # of terms of one sign, the bound of a long sum is a small share of it
        x.abs_(), wg.abs_(), wu.abs_()
    out = v.gated_ff(x, wg, wu, activation="silu", keep=True)
    want = R.gated(x, wg, wu, "silu")
    for got, w, b in zip(out, want[:3], want[3:]):
        near(got, w, b, dtype)
    for _ in range(8):
        for got, again in zip(out, v.gated_ff(x, wg, wu, activation="silu", keep=True)):
            assert torch.equal(got, again)
    assert v.device_errors() == 0
