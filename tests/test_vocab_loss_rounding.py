"""What rounding g to bf16 costs the vocabulary loss's gradients, for losses as
they come: targets drawn at random and from the model's own probabilities (a
trained model's, where the target's probability is not small), one dloss for
every row and another for each.

Tolerance.  A bf16 rounding is off by at most 2^-8 of the value, spread evenly:
a variance of at most 2^-16 / 3 of its square.  Each entry of g has one,
independent of the others', and each result one of its own:
  |error|^2 <= 2^-16 / 3 (sum over the terms of (g w)^2 + |dx|^2)
and likewise for dw.  (Each result by itself is held to test_vocab_loss.py's
bounds.)"""
import pytest
import torch

from tests.test_vocab_loss import Loss


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [False, True], ids=["mean", "weights"])
@pytest.mark.parametrize("drawn", [False, True], ids=["random", "drawn"])
@pytest.mark.parametrize("T,V,H,scale", [(300, 3000, 200, 2.0), (1001, 32001, 2000, 2.0), (1001, 32001, 2000, 4.0),
                                         (130, 40, 64, 3.0)])
def test_gradients(T, V, H, scale, drawn, weights):
    p = Loss(T, V, H, seed=3, scale=scale)
    x, w = p.x.double(), p.w.double()
    counts = p.target >= 0
    g = torch.softmax(x @ w.t(), 1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    if drawn:
        p.target.copy_(torch.where(counts, torch.multinomial(g, 1, generator=gen).squeeze(1), p.target))
    if weights:
        p.dloss.copy_(torch.rand(T, generator=gen, device="cuda") / T)
    else:
        p.dloss.fill_(1.0 / int(counts.sum()))
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()
    g[torch.arange(T, device="cuda"), torch.where(counts, p.target, 0)] -= 1
    g *= torch.where(counts, p.dloss.double(), 0.0)[:, None]
    gt = g.t().contiguous()
    for got, want, terms in ((p.dx, g @ w, (g * g) @ (w * w)), (p.dw, gt @ x, (gt * gt) @ (x * x))):
        error = (got.double() - want).pow(2).sum()
        assert error <= 2.0 ** -16 / 3 * (terms.sum() + want.pow(2).sum())
