"""Every kernel that the vocabulary loss can take, each at sizes that reach it:
the plan says which ones they are, so that a rule which moves the sizes to
other kernels fails here instead of leaving one without a test (tolerances:
test_vocab_loss.py's)."""
import ctypes

import pytest
import torch

from tests.test_vocab_loss import Loss
from warp_specialized_pipelined_amd import migemm

BAD = migemm.MIGEMM_ERR_INVALID_ARG


def test_info_refuses_what_is_not_a_loss_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_vocab_loss_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_vocab_loss_plan_get_info(p, ctypes.byref(info)) == BAD
    assert bytes(info) == bytes(ctypes.sizeof(info))


def taken(plan):
    """(tile of the logits forward, backward, of dx, its splits, of dw, its
    splits, pieces of the vocabulary)"""
    i = plan.info
    return ((i.forward_tile_m, i.forward_tile_n), (i.gradient_tile_m, i.gradient_tile_n),
            (i.dx_tile_m, i.dx_tile_n), i.dx_splits, (i.dw_tile_m, i.dw_tile_n), i.dw_splits, i.pieces)


ROWS, T64, T64x128, T128, T256 = (16, 32), (64, 64), (64, 128), (128, 128), (256, 256)

# Rows, vocabulary and hidden size end inside a tile and inside a K stage.
SIZES = [
    # 256 x 256 tiles: dx in one range of K, in a few, in 8 and more (whose
    # sums four waves join); one piece of the vocabulary and several, the last
    # one shorter; dw beside it in 128 x 128 tiles.
    ((3047, 2886, 3092), (T256, T256, T256, 1, T256, 1, 1)),
    ((660, 4129, 3617), (T128, T128, T256, 4, T256, 1, 1)),
    ((1025, 16001, 1000), (T128, T128, T256, 12, T256, 1, 1)),
    ((1001, 32001, 2000), (T256, T256, T256, 8, T256, 1, 1)),
    ((145, 39417, 1377), (T64x128, T64x128, T256, 32, T128, 1, 1)),
    ((6546, 40452, 2149), (T256, T256, T256, 1, T256, 1, 2)),
    ((2870, 87799, 143), (T128, T128, T256, 16, T256, 1, 2)),
    ((3001, 100001, 800), (T256, T256, T256, 16, T256, 1, 2)),
    ((8192, 100000, 700), (T256, T256, T256, 8, T256, 1, 4)),
    # one row
    ((1, 64984, 2729), (T256, T256, T128, 16, T128, 1, 1)),
    # dx in small tiles beside dw in large ones, and in other small ones
    ((940, 4925, 2444), (T128, T128, T128, 3, T256, 1, 1)),
    ((538, 3869, 3338), (T128, T128, T64x128, 1, T256, 1, 1)),
    ((1, 104410, 342), (T64x128, T64x128, T64x128, 64, T128, 1, 1)),
    ((1, 62704, 201), (T64x128, T64x128, T64, 64, T128, 1, 1)),
    # small tiles: alike for both, with split sums of either and of both, and
    # several pieces
    ((2735, 98394, 67), (T128, T128, T128, 16, T128, 1, 2)),
    ((2949, 828, 474), (T64x128, T64x128, T64x128, 1, T64x128, 4, 1)),
    ((2600, 200, 100), (T64, ROWS, T64, 1, T64, 12, 1)),
    ((600, 1000, 40), (T64, ROWS, T64, 4, T64, 2, 1)),
    ((300, 5000, 72), (T64x128, T64, T64, 16, T64, 1, 1)),
    ((17, 3000, 200), (ROWS, ROWS, T64, 12, T64, 1, 1)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size,kernels", SIZES, ids=["x".join(map(str, s)) for s, _ in SIZES])
def test_kernels(size, kernels):
    p = Loss(*size, seed=sum(size), skip=0.2 if size[0] > 2 else 0.0)
    assert taken(p.plan) == kernels
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()
    outs = (p.loss, p.dx, p.dw)
    want = [t.clone() for t in outs]
    # Rows that do not count may hold anything, and so may the workspace.
    dead = p.target < 0
    p.x[dead] = float("nan")
    p.dloss[dead] = float("inf")
    for t in outs:
        t.fill_(7)
    p.ws.fill_(0xFF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.forward(s)
    p.backward(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.gpu
def test_info_of_other_plans():
    p = Loss(300, 5000, 72, train=False)
    assert taken(p.plan) == (T64x128, (0, 0), (0, 0), 0, (0, 0), 0, 0) and p.plan.info.piece == 0
    assert p.plan.info.cu_count == torch.cuda.get_device_properties(0).multi_processor_count
    q = migemm.VocabLossPlan(4100, 100000, 64, x_rs=64, w_rs=64, dx_rs=64, dw_rs=64).info
    assert q.piece % 256 == 0 and (q.pieces - 1) * q.piece < 100000 <= q.pieces * q.piece
    info, lib = migemm.migemm_vocab_loss_info(), migemm.load()
    n = migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64)
    assert lib.gemm_vocab_loss_plan_get_info(n.handle, ctypes.byref(info)) == BAD
    assert lib.gemm_vocab_loss_plan_get_info(p.plan.handle, None) == BAD
