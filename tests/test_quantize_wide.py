"""Rows to 8 bits where more than 256 rows of 8193 to 16384 columns take four
waves with eight vectors a lane: both types, whole and partial last vectors, on
another stream and in a graph.  Codes and scales: test_quantize.py's definition."""
import pytest
import torch

from tests.test_quantize import E4M3, INT8, Rows

pytestmark = pytest.mark.gpu


def rows_of(rows, cols, q_type, pad=1):
    g = torch.Generator().manual_seed(rows * 5 + cols)
    x = torch.randn(rows, cols, generator=g)
    x[rows // 2] = 0
    x[:, cols - 1] *= 4  # the last column holds many rows' largest magnitude
    return Rows(x.bfloat16(), q_type, pad)


@pytest.mark.parametrize("rows,cols", [(300, 8193), (257, 8200), (257, 12001), (1000, 10007), (300, 14335),
                                       (300, 14337), (300, 16383), (300, 16384)])
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
@pytest.mark.parametrize("pad", [0, 1])
def test_rows(rows, cols, q_type, pad):
    p = rows_of(rows, cols, q_type, pad)
    assert (p.plan.info.waves, p.plan.info.vectors) == (4, 8)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("rows,cols,shape", [(256, 12001, (16, 2)), (257, 12001, (4, 8)), (257, 16384, (4, 8)),
                                             (257, 16385, (16, 4)), (257, 8192, (4, 4))])
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
def test_kernels_and_runs_on_streams_and_in_a_graph(rows, cols, shape, q_type):
    p = rows_of(rows, cols, q_type)
    assert (p.plan.info.waves, p.plan.info.vectors) == shape
    p.run()
    torch.cuda.synchronize()
    p.check()
    q, scale = p.q_full.clone(), p.scale.clone()

    def spoil():
        p.q_full[:, :cols] = 3
        p.scale.fill_(3)
        torch.cuda.synchronize()

    spoil()
    p.run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(p.q_full, q) and torch.equal(p.scale, scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(3):
        spoil()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.q_full, q) and torch.equal(p.scale, scale)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.q_full, q)


def test_rows_that_hold_no_number():
    for q_type in (INT8, E4M3):
        p = rows_of(300, 12001, q_type)
        p.x[3, 12000] = float("nan")
        p.x[299, 0] = float("inf")
        p.run()
        torch.cuda.synchronize()
        q, scale = p.q.float().cpu(), p.scale.cpu()
        assert torch.isnan(scale[[3, 299]]).all() and (q[[3, 299]] == 0).all()
        assert torch.isfinite(scale).sum() == 298
        p.x[3], p.x[299] = 0, 0
        p.run()
        torch.cuda.synchronize()
        p.check()
