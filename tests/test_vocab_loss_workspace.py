"""The vocabulary loss's workspace is within what its description states."""
import pytest

from warp_specialized_pipelined_amd import migemm

MiB = 1 << 20


def tiles(rows, cols, tile_m, tile_n):
    return -(-rows // tile_m) * -(-cols // tile_n) * tile_m * tile_n


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", [(1, 100, 64), (1001, 32001, 2000), (2048, 131072, 4096), (8192, 131072, 4096),
                                   (8192, 100000, 700), (16400, 20000, 24), (70000, 50000, 64), (262144, 32000, 64),
                                   (262145, 1025, 64), (600000, 5000, 64), (1 << 20, 3000, 64), (0, 300, 40)])
def test_within_the_statement(T, V, H):
    ld = -(-H // 8) * 8
    p = migemm.VocabLossPlan(T, V, H, x_rs=ld, w_rs=ld, dx_rs=ld, dw_rs=ld)
    i = p.info
    width = min(i.piece, -(-V // 64) * 64)
    assert i.piece <= 1024 or 2 * T * i.piece <= 512 * MiB
    g = 2 * T * (width + 64)
    rows = T * (2 * -(-H // 64) * 64 + 16)                      # x, lse, dloss, target and the row's number
    dx, dw = (4 * tiles(r, H, m, n) for r, m, n in
              ((T, i.dx_tile_m, i.dx_tile_n), (min(i.piece, V), i.dw_tile_m, i.dw_tile_n)))
    alone = i.dx_splits == 1 and i.pieces == 1 and i.dx_tile_m < 256   # a workgroup finishes its tile of dx
    sums = (0 if alone else i.dx_splits * dx) + (i.dw_splits * dw if i.dw_splits > 1 else 0)
    assert i.dx_splits == 1 or i.dx_splits * 4 * T * H <= 512 * MiB
    assert i.dw_splits == 1 or i.dw_splits * 4 * min(i.piece, V) * H <= 512 * MiB
    forward = 8 * min(T, 16384) * -(-V // 16) + 4 * min(T, 16384)
    assert p.workspace_size <= max(forward, 256 + g + rows + sums + 8 * 256)
