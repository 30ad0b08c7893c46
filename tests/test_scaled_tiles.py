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


@pytest.mark.gpu
def test_more_tiles_than_a_launch_has_threads_for():
    """8400 x 4190000 results of a short sum: their 64 x 64 tiles of 256
    threads come in more than one launch.  Whole numbers: exact."""
    M, N, K = 8400, 4_190_000, 16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB")
    a = torch.ones((M, K), device="cuda").to(torch.float8_e4m3fn)
    col = torch.arange(N, device="cuda")
    value = torch.tensor([0.0, 1.0, -1.0, 2.0], device="cuda")
    b = torch.ones((N, K), device="cuda")
    b[:, 5] = value[col % 4]
    b[:, 15] = value[(col // 7) % 4]
    total = b.sum(1)
    b = b.to(torch.float8_e4m3fn)
    sa = 2.0 ** (torch.arange(M, device="cuda") % 5).float()
    sb = torch.ones(N, device="cuda")
    sb[::3] = 2.0
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    plan = migemm.ScaledPlan(M, N, K, a_rs=K, b_cs=K, d_rs=N)
    assert plan.workspace_size == 0
    plan.run(a, sa, b, sb, d)
    torch.cuda.synchronize()
    for f in range(0, M, 60):
        want = (total * sb)[None, :] * sa[f:f + 60, None]
        assert torch.equal(d[f:f + 60], want.bfloat16()), f


# 128 x 128 tiles two a compute unit: K of a few stages and of many, an odd
# number and an even one, its end inside one; whole and with split sums.
PAIRS = [(2773, 2191, 552), (1500, 3001, 385), (3000, 2100, 641), (1200, 2000, 9001), (542, 8056, 7030),
         (2001, 2745, 3100)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_two_tiles_a_compute_unit(M, N, K):
    p = Scaled(M, N, K, seed=M + N + K)
    p.a[M // 2, K - 1] = float("nan")
    p.run()
    torch.cuda.synchronize()
    nan = torch.isnan(p.d.float())
    assert nan[M // 2].all() and int(nan.sum()) == N
    p.a[M // 2, K - 1] = 0.0
    p.run()
    torch.cuda.synchronize()
    p.check()
    first = p.d.clone()
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.d, first)
