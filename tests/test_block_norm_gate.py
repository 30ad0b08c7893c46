"""How near the block norm's gate is to the sigmoid, seen through rstd, which is
fp32 and of one value a row: with one column, no norm behind the block and a
residual scale of 0, rstd = 1 / sqrt((sigmoid(z) x)^2 + eps).

Its error in units of U = 2^-24: the gate's exponential one unit in the last
place, 2, and what is put back of its argument rounded once, 1 (what remains of
the argument's rounding is of second order: (|z| 2^-24)^2); the sum 1, its
reciprocal 1 and, for z < 0, the product 1; times x 1, and times branch and onto
0, exact: 7.  Its square twice that and 1, the sum's rounding with eps 1; the
root halves that to 8, and its own is a unit in the last place, 2: 10.  One of
10 for the second order."""
import pytest
import torch

from tests.test_block_norm import Block

U = 2.0 ** -24
BOUND = 11 * U
EPS = 1e-30


def gates():
    """Every bf16 z of magnitudes from 2^-8 to 87, below which exp(-|z|) is no subnormal."""
    bits = torch.arange((127 - 8) << 7, (127 + 7) << 7, dtype=torch.int32)
    z = bits.to(torch.int16).view(torch.bfloat16)
    z = z[z.float() <= 87]
    return torch.cat([z, -z])


def operands():
    z = gates().double()
    s = torch.where(z < 0, torch.exp(z) / (1 + torch.exp(z)), 1 / (1 + torch.exp(-z)))
    x = torch.exp2(-torch.log2(s).round()).bfloat16()      # so that h is between 0.7 and 1.5
    h = s * x.double()
    assert ((h > 0.7) & (h < 1.5)).all()
    return gates(), x, (h * h + EPS).rsqrt()


def test_an_exponential_of_a_rounded_argument_is_outside_the_bound():
    """What the product with log2 e rounds off, not put back (the rest in 64 bits)."""
    z, x, want = operands()
    m = z.float().abs()
    e = torch.exp2(-(m * torch.tensor(1.44269502)).double())
    s = torch.where(z.double() < 0, e, 1.0) / (1 + e)
    off = (((s * x.double()) ** 2 + EPS).rsqrt() / want - 1).abs()
    assert off.max() > 2 * BOUND and (off > BOUND).sum() > 100


@pytest.mark.gpu
def test_gate():
    z, x, want = operands()
    p = Block(len(z), 1, post=False, branch=1.0, residual=0.0)
    p.z[:, 0], p.x[:, 0] = z.cuda(), x.cuda()
    import tests.test_block_norm as module
    eps, module.EPS = module.EPS, EPS
    try:
        p.make_plan()
    finally:
        module.EPS = eps
    p.forward()
    torch.cuda.synchronize()
    off = (p.rstd.double().cpu() / want - 1).abs()
    print("largest error %.1f units of 2^-24" % (off.max().item() / U))
    assert (off <= BOUND).all(), (off.max().item() / U, z[off.argmax()].item())
