"""The scaled product's smaller tiles and its split sums, at the sizes where
they begin, end and have parts (tolerances: test_scaled.py's)."""
import pytest
import torch

from tests.test_scaled import Scaled
from warp_specialized_pipelined_amd import migemm

# Tiles of 64 and 128, one to either side; K of one to many 128-byte stages,
# with 1 to 15 bytes of a 16-byte chunk left over; long K with few tiles
# (split), and splits that do not divide it.
SHAPES = [(65, 63, 257), (128, 128, 384), (129, 127, 511), (64, 512, 1025), (100, 300, 3001),
          (127, 3000, 385), (192, 320, 16384), (26, 386, 10623), (142, 752, 13655), (108, 1100, 14436),
          (300, 2000, 8191), (1000, 1100, 300), (513, 4097, 1000), (2000, 65, 9001), (1030, 1030, 4111),
          (4000, 70, 200), (3000, 130, 255), (700, 129, 256), (17, 16, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    p = Scaled(M, N, K, seed=M + 5 * N + 11 * K)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(26, 386, 10623), (142, 752, 13655), (300, 1000, 1000), (1000, 1100, 200)])
def test_runs_agree_on_streams_and_in_a_graph(M, N, K):
    p = Scaled(M, N, K, seed=6)
    p.run()
    torch.cuda.synchronize()
    want = p.d.clone()

    def same():
        torch.cuda.synchronize()
        ok = torch.equal(p.d, want)
        p.d.fill_(7)
        if p.ws is not None:
            p.ws.fill_(0xFF)
        torch.cuda.synchronize()
        return ok

    assert same()
    p.run(torch.cuda.Stream())
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(3):
        graph.replay()
        assert same()
        p.run()
        assert same()


@pytest.mark.gpu
def test_a_nan_stays_in_its_row_and_column():
    """Also from the storage beside a row's last K, and with split sums."""
    for M, N, K in ((142, 752, 13655), (300, 1000, 1001), (100, 200, 129)):
        p = Scaled(M, N, K, seed=2)
        p.a[M // 2, K - 1] = float("nan")
        p.b[N // 3, 0] = float("nan")
        p.run()
        torch.cuda.synchronize()
        nan = torch.isnan(p.d.float()).cpu()
        want = torch.zeros(M, N, dtype=torch.bool)
        want[M // 2, :] = True
        want[:, N // 3] = True
        assert torch.equal(nan, want), (M, N, K)


@pytest.mark.gpu
def test_a_plan_with_split_sums_needs_its_workspace():
    p = Scaled(142, 752, 13655)
    assert p.plan.workspace_size > 0
    lib, plan = migemm.load(), p.plan.handle
    a = [p.a.data_ptr(), p.sa.data_ptr(), p.b.data_ptr(), p.sb.data_ptr(), p.d.data_ptr()]
    assert lib.gemm_scaled_run(plan, *a, None, None) == migemm.MIGEMM_ERR_INVALID_ARG
    assert lib.gemm_scaled_run(plan, *a, p.ws.data_ptr() + 16, None) == migemm.MIGEMM_ERR_MISALIGNED


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(4000, 3000, 1000), (1500, 6000, 513), (2900, 4100, 2057), (193 * 16, 8192, 300),
                                   (5000, 5000, 257)])
def test_large_tiles_of_both_heights(M, N, K):
    """192 and 256 rows a tile, with rows, columns and K past the last whole one."""
    p = Scaled(M, N, K, seed=M + N + K)
    p.run()
    torch.cuda.synchronize()
    p.check()
