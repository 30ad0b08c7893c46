"""The scaled product's rounding, as its description states it: up to K = 256
exact products in fp32 sums; above, each octet of products (k = 8 i .. 8 i + 7)
cut to multiples of 2^-13 of its largest one's power of two.  Rows with
outliers, products that cancel, and codes of every size, in every kind of tile
(the bounds are test_scaled_kernels.py's)."""
import pytest
import torch

from tests.test_scaled import Scaled
from tests.test_scaled_kernels import check

# (rows, columns, K) and the tile and LDS stages that take it.
SIZES = [
    ((17, 33, 257), (16, 16, 0)), ((17, 33, 4097), (16, 16, 0)), ((1, 4174, 288), (16, 32, 0)),
    ((127, 3001, 385), (32, 32, 0)), ((1001, 1101, 300), (64, 32, 0)), ((1001, 1003, 1001), (64, 64, 4)),
    ((142, 752, 13655), (64, 128, 3)), ((513, 4097, 1001), (64, 128, 3)), ((424, 6578, 7971), (128, 128, 4)),
    ((2773, 2191, 552), (128, 128, 2)), ((2900, 4100, 2057), (256, 256, 2)), ((790, 10137, 537), (192, 256, 2)),
    ((16, 1001, 256), (16, 64, 0)), ((700, 129, 256), (64, 64, 2)), ((300, 500, 97), (64, 64, 2)),
]


def to_codes(t):
    return t.clamp(-448, 448).to(torch.float8_e4m3fn)


def channels(M, N, K, g):
    """A few channels of a at 448, the others 400 times smaller."""
    a = torch.randn(M, K, generator=g)
    a[:, ::61] = torch.where(torch.rand(M, a[:, ::61].shape[1], generator=g) < 0.5, -448.0, 448.0)
    return a, torch.randn(N, K, generator=g) * 60


def pairs(M, N, K, g):
    """Two products of 448 x 448 that cancel in every fifth octet."""
    a = torch.randn(M, K, generator=g) * 4
    b = torch.randn(N, K, generator=g)
    for k in range(0, K - 7, 40):
        a[:, k] = a[:, k + 5] = b[:, k] = 448.0
        b[:, k + 5] = -448.0
    return a, b


def every_code(M, N, K, g):
    """Codes of every size, subnormal ones among them."""
    def draw(n):
        c = torch.randint(0, 256, (n, K), generator=g, dtype=torch.uint8)
        c[(c & 127) == 127] = 0     # (no NaN)
        return c.view(torch.float8_e4m3fn).float()
    return draw(M), draw(N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [channels, pairs, every_code])
@pytest.mark.parametrize("size,tile", SIZES, ids=["x".join(map(str, s)) for s, _ in SIZES])
def test_within_the_stated_bound(size, tile, kind):
    p = Scaled(*size, seed=1)
    i = p.plan.info
    assert (i.tile_m, i.tile_n, i.lds_stages) == tile and i.exact == (size[2] <= 256)
    a, b = kind(*size, torch.Generator().manual_seed(sum(size)))
    p.a.copy_(to_codes(a))
    p.b.copy_(to_codes(b))
    p.run()
    torch.cuda.synchronize()
    check(p)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(17, 33, 256), (16, 1001, 255), (700, 129, 256), (300, 500, 97)])
def test_short_sums_keep_what_stands_beside_a_cancelling_pair(size):
    """Exact: six products of 7 beside 448 x 448 - 448 x 448 in an octet."""
    M, N, K = size
    p = Scaled(M, N, K)
    for at in (0, 8 * (K // 16), 8 * (K // 8 - 1)):
        p.a.copy_(torch.zeros(M, K).to(torch.float8_e4m3fn))
        p.b.copy_(torch.zeros(N, K).to(torch.float8_e4m3fn))
        p.a[:, at:at + 8] = 7.0
        p.b[:, at:at + 8] = 1.0
        p.a[:, at + 1] = p.a[:, at + 6] = p.b[:, at + 1] = 448.0
        p.b[:, at + 6] = -448.0
        p.sa.fill_(1.0)
        p.sb.fill_(1.0)
        p.run()
        torch.cuda.synchronize()
        assert (p.d.float() == 42.0).all(), at


@pytest.mark.gpu
@pytest.mark.parametrize("size", [s for s, _ in SIZES if s[2] > 256])
def test_longer_sums_lose_only_within_the_octet(size):
    """The same pair in one octet, the products of 7 in every other one: those
    are kept.  They add up below 2^11, so no fp32 sum of them rounds, and the
    pair is gone (to 200704 2^-23 a rounding) before or after them."""
    M, N, K = size
    p = Scaled(M, N, K)
    p.sa.fill_(1.0)
    p.sb.fill_(1.0)
    p.a.copy_(torch.zeros(M, K).to(torch.float8_e4m3fn))
    p.b.copy_(torch.zeros(N, K).to(torch.float8_e4m3fn))
    for k in range(8, min(K, 1600), 8):
        p.a[:, k], p.b[:, k] = 7.0, 1.0
    whole = 7.0 * len(range(8, min(K, 1600), 8))
    p.a[:, 1] = p.a[:, 6] = p.b[:, 1] = 448.0
    p.b[:, 6] = -448.0
    p.run()
    torch.cuda.synchronize()
    assert ((p.d.float() - whole).abs() <= 2.0 ** -8 * whole + 200 * 200704 * 2.0 ** -23).all()
