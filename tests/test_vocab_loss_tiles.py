"""The vocabulary loss's smaller tiles, split products and row shares, at the
sizes where they begin, end and have parts (tolerances: test_vocab_loss.py's)."""
import pytest
import torch

from tests.test_vocab_loss import Loss

# Rows that the workgroups that copy them share unevenly, some getting none
# (1282, 2049); tiles of 64 and 128 and one to either side; few rows with a
# long vocabulary, many with a short one (K split); odd hidden sizes.
SHAPES = [(1282, 300, 40), (2049, 130, 65), (1030, 100, 64), (63, 64, 129), (65, 129, 63), (128, 127, 1000),
          (5, 20000, 70), (1, 12804, 300), (2600, 200, 100), (3000, 129, 333), (300, 5000, 72), (197, 1327, 2040),
          (700, 3000, 130), (2949, 828, 474)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_loss_and_gradients(T, V, H):
    p = Loss(T, V, H, seed=T + 2 * V + 3 * H)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", [(40, 3000, 100), (1282, 200, 64), (20, 20000, 70)])
def test_rows_that_hold_anything_reach_nothing(T, V, H):
    p, q = Loss(T, V, H, seed=5), Loss(T, V, H, seed=5)
    dead = p.target < 0
    assert dead.any()
    p.x[dead] = float("nan")
    q.x[dead] = 0
    p.dloss[dead] = float("inf")
    for m in (p, q):
        m.forward()
        m.backward()
    torch.cuda.synchronize()
    assert torch.equal(p.dw, q.dw) and torch.equal(p.dx, q.dx)
    assert (p.dx[dead] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", [(300, 700, 100), (33, 5000, 64)])
def test_a_mean_loses_nothing_to_its_factor(T, V, H):
    """The same dloss in every row is a factor of the gradients: a power of
    two scales them exactly, and their error against 64 bits stays that of
    one rounding (2^-8 at most, 2^-9 on average) whatever the factor is."""
    p, q = Loss(T, V, H, seed=7), Loss(T, V, H, seed=7)
    p.dloss.fill_(1.0 / 3)
    q.dloss.fill_(2.0 / 3)
    for m in (p, q):
        m.forward()
        m.backward()
    torch.cuda.synchronize()
    assert torch.equal(p.dx.float() * 2, q.dx.float()) and torch.equal(p.dw.float() * 2, q.dw.float())
    x, w = p.x.double(), p.w.double()
    counts = p.target >= 0
    g = torch.softmax(x @ w.t(), 1)
    g[torch.arange(T, device="cuda"), torch.where(counts, p.target, 0)] -= 1
    g *= torch.where(counts, p.dloss.double(), 0.0)[:, None]
    for got, want in ((p.dx, g @ w), (p.dw, g.t().contiguous() @ x)):
        # half a step of 2^-8, uniformly spread: 2^-8 / sqrt(3) of the norm at
        # most, over the rounding of g's small part
        assert (got.double() - want).norm() <= 2.0 ** -8 / 3 ** 0.5 * want.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("dloss", [[0.0, 0.0, 0.0], [float("nan"), 1.0, 2.0], [float("inf"), 1.0, 2.0], [1e-42, 2e-42, 0.0],
                                   [3e38, 1.0, -2e38]])
def test_factors_of_every_kind(dloss):
    p = Loss(3, 200, 64, seed=3, skip=0.0)
    p.dloss.copy_(torch.tensor(dloss))
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    dx = p.dx.float()
    for r, d in enumerate(dloss):
        if d != d or abs(d) == float("inf"):
            assert not torch.isfinite(dx[r]).any()
        elif d == 0:
            assert (dx[r] == 0).all()
        elif abs(d) > 1e-30:
            x, w = p.x[r].double(), p.w.double()
            g = torch.softmax(w @ x, 0)
            g[p.target[r]] -= 1
            want = d * (g @ w)
            fits = want.abs() < 3.3e38
            err = (dx[r].double() - want).abs()
            assert (err[fits] <= 2.0 ** -6 * d.__abs__() * (g.abs() @ w.abs())[fits]).all()
