"""Every kernel that an int8 product and a checkpoint's gradient can take, each
at sizes that reach it, odd ones: the plan says which one it is, so that a rule
which moves the sizes to another kernel fails here instead of leaving one
without a test.  Tolerances: test_int8.py's and test_checkpoint.py's."""
import pytest
import torch

from tests.test_checkpoint import BF16, FP32, Checkpoint
from tests.test_int8 import Int8

# (rows, columns, stages of K in LDS, K split) of a kernel, and sizes that reach it.
INT8 = [
    ((256, 256, 2, False), [(2900, 4100, 2057), (884, 15509, 1752)]),
    ((192, 256, 2, False), [(1426, 6120, 397), (1643, 5325, 519)]),
    ((16, 16, 0, False), [(17, 33, 4001), (1, 16, 3631)]),
    ((16, 32, 0, False), [(36, 1454, 4187), (33, 1806, 4010)]),
    ((32, 32, 0, False), [(127, 3001, 385), (1, 17, 18), (5516, 17, 16)]),
    ((64, 32, 0, False), [(40, 9675, 18), (5485, 79, 19)]),
    ((64, 64, 4, False), [(1001, 1003, 1001), (9, 16723, 71)]),
    ((64, 64, 4, True), [(2205, 18, 13802), (21, 2310, 13919)]),
    ((64, 128, 3, False), [(941, 3813, 227), (149, 12849, 16)]),
    ((64, 128, 3, True), [(34, 2802, 15899), (68, 1712, 13638)]),
    ((128, 128, 2, False), [(2773, 2191, 552), (8362, 403, 19)]),
    ((128, 128, 2, True), [(5933, 42, 15399), (1200, 2000, 9001)]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,size", [(k, s) for k, sizes in INT8 for s in sizes])
def test_int8_kernel(kernel, size):
    M, N, K = size
    p = Int8(M, N, K, seed=M + 2 * N + 3 * K)
    i = p.plan.info
    assert (i.tile_m, i.tile_n, i.lds_stages, i.splits > 1) == kernel
    assert i.cu_count == torch.cuda.get_device_properties(0).multi_processor_count
    p.run()
    torch.cuda.synchronize()
    p.check()
    first = p.d.clone()
    p.d.fill_(7)
    if p.ws is not None:
        p.ws.fill_(0xFF)
    p.run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(p.d, first)


# (rows, columns of dw, stages in LDS, tokens split) and (tokens, columns, dy's columns).
KEPT = [
    ((64, 64, 4, False), [(1, 17, 19), (70, 300, 1001)]),
    ((64, 64, 4, True), [(1421, 18, 19), (20001, 301, 203)]),
    ((128, 128, 3, False), [(1, 13856, 194), (333, 1001, 4101)]),
    ((128, 128, 3, True), [(4072, 73, 4145), (6725, 3440, 65)]),
    ((192, 256, 3, False), [(469, 692, 11186), (1001, 2000, 5000)]),
    ((192, 256, 3, True), [(10096, 5901, 164), (10906, 6753, 147)]),
    ((256, 256, 3, False), [(1236, 11522, 1063), (1328, 15398, 804)]),
    ((256, 256, 3, True), [(13211, 8270, 490)]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,size", [(k, s) for k, sizes in KEPT for s in sizes])
@pytest.mark.parametrize("dw_type,accumulate", [(BF16, False), (FP32, False), (FP32, True)])
def test_gradient_kernel(kernel, size, dw_type, accumulate):
    tokens, cols, out_cols = size
    p = Checkpoint(tokens, cols, out_cols, dw_type, accumulate, seed=tokens + 2 * cols + 3 * out_cols)
    i = p.plan.info
    # (fp32 sums cost more to store: a size may then take another split.)
    if dw_type == BF16:
        assert (i.tile_m, i.tile_n, i.lds_stages, i.splits > 1) == kernel
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    p.check_gradient()
    first = p.dw.clone()
    if accumulate:
        p.dw.copy_(p.before)
    if p.ws is not None:
        p.ws.fill_(0xFF)
    p.gradient(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(p.dw, first)
