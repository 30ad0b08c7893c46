"""Where the block's operators leave fp32's range on the way to a result that
bf16 or 8 bits could hold: as the header says, and only in the rows and columns
concerned."""
import pytest
import torch

from tests.test_block_norm import BF16, E4M3, INT8, Block, check
from tests.test_int8 import Int8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (40, 300, 200), (300, 300, 4096), (30, 200, 9000), (2900, 4100, 200)])
def test_int8_scales_are_taken_in_their_order(M, N, K):
    p = Int8(M, N, K, seed=3, low=1, bias=False)
    p.sa.fill_(2.0 ** 100)
    p.sb.fill_(2.0 ** -100)
    p.run()
    torch.cuda.synchronize()
    p.check()                                       # sum 2^100 is far below 2^128
    p.sa[M // 2] = 2.0 ** 127                       # times a sum of 2 or more
    p.a[M // 2], p.b[:, 0] = 127, 127
    p.run()
    torch.cuda.synchronize()
    d = p.d.float()
    assert torch.isinf(d[M // 2]).all() and torch.isfinite(d).sum() == (M - 1) * N


@pytest.mark.parametrize("rows,cols", [(9, 500), (300, 8191), (40, 16382)])
def test_block_norm_where_h_times_its_weight_has_no_fp32(rows, cols):
    for y_type in (BF16, E4M3, INT8):
        p = Block(rows, cols, y_type, post=False, gate=False, seed=7)
        p.weight[5] = 2.0 ** 100
        p.x[:, 5], p.r[:, 5] = 1.0, 0.0
        p.x[4], p.r[4] = 0.0, 0.0
        p.x[4, 5] = 2.0 ** 40                       # h * weight: 2^139.6
        p.forward()
        torch.cuda.synchronize()
        if y_type == BF16:                          # y = sqrt(cols) 2^100 there: formed from n = h rstd
            check(p)
            continue
        scale, y = p.scale.cpu(), p.y.float().cpu()
        assert not torch.isfinite(scale[4]) and torch.isfinite(scale).sum() == rows - 1
        if y_type == INT8:
            assert torch.isnan(scale[4]) and (y[4] == 0).all()
        p.x[4] = 0
        p.forward()
        torch.cuda.synchronize()
        check(p)
