"""The block's operators on rows far apart, up to the longest strides that a plan
takes: what comes out is what close rows give, bit for bit (a plan's choice goes
by sizes, not by strides)."""
import pytest
import torch

from tests.test_block_norm import Block
from tests.test_checkpoint import BF16, FP32, Checkpoint
from tests.test_int8 import Int8
from tests.test_operators_past_32_bits import need
from tests.test_quantize import E4M3, Rows
from warp_specialized_pipelined_amd import migemm

pytestmark = pytest.mark.gpu

BAND = 0x7FFFFFF0 - 1024  # bytes that 256 rows of a product's matrix may span


def apart(t, ld, copy=True):
    """t's rows ld elements apart; what lies between is left as it is."""
    full = torch.empty((t.shape[0], ld), dtype=t.dtype, device="cuda")
    v = full[:, :t.shape[1]]
    if copy:
        v.copy_(t)
    return v


def longest(size, rows):
    """The longest stride, in elements, that a product's matrix may have."""
    return BAND // 256 // 16 * 16 // size


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [(1, 40, 200), (40, 33, 300), (300, 300, 1000), (30, 300, 9000), (300, 500, 200),
                                   (520, 800, 520)])
def test_int8(M, N, K):
    need(40)
    p = Int8(M, N, K, seed=M)
    p.run()
    a, b, d = apart(p.a, longest(1, M)), apart(p.b, longest(1, N)), apart(p.d, longest(2, M), False)
    plan = migemm.Int8Plan(M, N, K, a_rs=a.stride(0), b_cs=b.stride(0), d_rs=d.stride(0))
    plan.run(a, p.sa, b, p.sb, p.bias, d, p.ws)
    torch.cuda.synchronize()
    p.check()
    assert same(d, p.d)


@pytest.mark.parametrize("tokens,cols,out_cols", [(1, 17, 19), (130, 300, 333), (1421, 18, 19), (257, 520, 600),
                                                  (469, 692, 1186)])
@pytest.mark.parametrize("dw_type,accumulate", [(BF16, False), (FP32, True)], ids=["bf16", "accumulate"])
def test_checkpoint(tokens, cols, out_cols, dw_type, accumulate):
    need(60)
    p = Checkpoint(tokens, cols, out_cols, dw_type, accumulate, seed=tokens)
    p.pack()
    p.gradient()
    dy = apart(p.dy, longest(2, tokens))
    dw = apart(p.before if accumulate else p.dw, longest(4 if dw_type == FP32 else 2, out_cols), accumulate)
    x = apart(p.x, 1 << 23)
    plan = migemm.CheckpointPlan(tokens, cols, x_rs=x.stride(0), out_cols=out_cols, dy_rs=dy.stride(0),
                                 dw_rs=dw.stride(0), dw_type=dw_type, accumulate=accumulate)
    kept = torch.full_like(p.kept, 0x7E)
    plan.pack(x, kept)
    plan.weight_gradient(dy, kept, dw, p.ws)
    torch.cuda.synchronize()
    assert same(kept, p.kept) and same(dw, p.dw)
    plan.unpack(kept, x)
    torch.cuda.synchronize()
    assert torch.equal(x.double().cpu(), p.value())


@pytest.mark.parametrize("rows,cols", [(5, 511), (5, 2048), (5, 8001), (5, 16383)])
def test_rows(rows, cols):
    """Strides past 2^32 bytes."""
    need(150)
    p = Block(rows, cols, seed=rows)
    p.forward()
    p.backward()
    q = Rows(p.x, E4M3)
    q.run()
    torch.cuda.synchronize()
    far = (1 << 31) + 64
    x = apart(p.x, far)
    codes, scale = apart(q.q.view(torch.int8), far, False), torch.empty_like(q.scale)
    migemm.QuantizePlan(rows, cols, E4M3, x_rs=far, q_rs=far).run(x, codes, scale)
    torch.cuda.synchronize()
    assert same(codes, q.q) and same(scale, q.scale)
    del codes
    h = apart(p.h, far, False)
    rs = {k + "_rs": getattr(p, k).stride(0) for k in ("z", "r", "y", "dy", "dh", "dr", "dz")}
    plan = migemm.BlockNormPlan(rows, cols, 1e-5, branch_scale=p.branch, residual_scale=p.residual, x_rs=far, h_rs=far,
                                dx_rs=far, **rs)
    y, rstd, post_rstd = torch.empty_like(p.fulls["y"])[:, :cols], torch.empty_like(p.rstd), torch.empty_like(p.rstd)
    plan.run(x, p.z, p.r, p.post_weight, p.weight, h, y, None, post_rstd, rstd)
    torch.cuda.synchronize()
    assert same(h, p.h) and same(y, p.y) and same(rstd, p.rstd) and same(post_rstd, p.post_rstd)
    dx, dz, dr, dw, dpw = (t.clone() for t in (p.dx, p.dz, p.dr, p.dweight, p.dpost_weight))
    plan.run_backward(p.dy, p.dh, x, p.z, h, p.post_weight, p.weight, post_rstd, rstd, x, p.dz, p.dr, p.dpost_weight,
                      p.dweight, p.ws)
    torch.cuda.synchronize()
    for a, b in ((x, dx), (p.dz, dz), (p.dr, dr), (p.dweight, dw), (p.dpost_weight, dpw)):
        assert same(a, b)
