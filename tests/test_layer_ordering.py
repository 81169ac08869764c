"""Codes of 8-bit activations that one lane of a warp fetches and others read
(the gradient of rows that are not whole 16-byte accesses): the order of the
reads and of the copies around them."""
import os

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "collective_reduction_virtual_gb300", "csrc")


def test_codes_read_across_lanes_lie_between_warp_barriers():
    # a wait covers a thread's own copies and a shuffle orders no memory: a warp barrier stands
    # between the copies' arrival and the reads, and between the reads and the slot's next copies
    src = open(os.path.join(CSRC, "norm_rows.cuh")).read()
    read = src.index("from -= t.lane", src.index("vc_norm_grad_rows"))
    arrival, refill = src.rindex("fetch_wait<", 0, read), src.index("fetch(s);", read)
    assert "KEPT && A < E) __syncwarp();" in src[arrival:read]
    assert "KEPT && A < E) __syncwarp();" in src[read:refill]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,ld", [(torch.bfloat16, 1), (torch.bfloat16, 2), (torch.float32, 1)])
@pytest.mark.parametrize("n,d", [(5000, 300), (3001, 998), (2500, 2050), (1300, 6002), (1201, 12290)])
def test_every_row_meets_its_own_codes(dtype, ld, n, d):
    # scales and gradients of 1, so that a column's sum over the rows is that of its codes: whole
    # numbers below 2^24, exact in any order, and wrong if any row met another's codes
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    width = (d + 15) // 16 * 16
    codes = torch.randint(-127, 128, (n, width), generator=g, device="cuda", dtype=torch.int8)
    codes[:, d:] = 0
    kept = vc.Checkpoint8(codes, torch.ones(n, -(-d // 128), device="cuda"), torch.Size((n, d)))
    grad = torch.ones(n * (d + ld), dtype=dtype, device="cuda").view(n, d + ld)[:, :d]
    rstd = torch.ones(n, device="cuda")
    for _ in range(3):
        _, dw, db = vc.layer_norm_backward_checkpoint8(grad, kept, rstd)
        assert torch.equal(dw.double(), codes[:, :d].double().sum(0))
        assert (db == n).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pad,at", [(torch.bfloat16, 0, 0), (torch.bfloat16, 2, 2), (torch.bfloat16, 1, 1),
                                          (torch.float32, 0, 0), (torch.float32, 1, 1)])
@pytest.mark.parametrize("d", [64, 128, 256, 512, 1024, 2048, 4096, 8192, 8704, 12288, 16384])
def test_copies_land_in_their_own_slots(dtype, pad, at, d):
    # codes and gradients that name their place among the columns that a warp copies: a copy that
    # landed in another slot would bring another column's number
    from collective_reduction_virtual_gb300 import build
    build.build()
    import collective_reduction_virtual_gb300 as vc
    n = 3
    col = torch.arange(d, device="cuda")
    for code in (col // 8 % 128, col // 1024 % 128, (col + col // 128) % 113):
        codes = code.to(torch.int8).repeat(n, 1)
        kept = vc.Checkpoint8(codes, torch.ones(n, -(-d // 128), device="cuda"), torch.Size((n, d)))
        flat = torch.zeros(n * (d + pad) + at, dtype=dtype, device="cuda")
        grad = flat[at:].view(n, d + pad)[:, :d]
        grad.copy_(1 + (col // 32 % 64) + torch.arange(n, device="cuda")[:, None])
        x = flat.clone()[at:].view(n, d + pad)[:, :d]
        x.copy_(code)
        mean, rstd = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
        total, want = grad.double().sum(0), (grad.double() * code).sum(0)
        for got in (vc.layer_norm_backward_checkpoint8(grad, kept, rstd),
                    vc.layer_norm_backward(grad, x, mean, rstd)):
            assert torch.equal(got[1].double(), want) and torch.equal(got[2].double(), total)
