"""What examples/eight_bit_block.py serves, step by step in 64 bits: each step is
compared with its definition on what the step before it left, so that a scale, a
bias or a row out of place shows wherever it stands.  Codes are the definition's
(test_quantize.py), the products' sums exact (test_int8.py), the norm's rows as
test_block_norm.py has them.

The weights' codes and those rows make the whole differ from fp32 by what 8 bits
cost: with the error of each of the four roundings measured from the codes
themselves, relative to what was rounded, and taken for independent, the result
is off by the root of the sum of their squares; twice that is allowed, and 2^-7
for the bf16 values between."""
import types

import pytest
import torch

from tests import test_block_norm
from tests.test_block_example import example  # noqa: F401 (a fixture)
from tests.test_quantize import INT8, TOP

pytestmark = pytest.mark.gpu


def check_codes(x, q, scale):
    x, top = x.double(), TOP[INT8]
    largest = x.abs().amax(1)
    want = torch.round(x * top / torch.where(largest > 0, largest, 1.0)[:, None])
    assert torch.equal(q.double(), want)
    assert ((scale.double() - largest / top).abs() <= 2.0 ** -24 * largest / top + 2.0 ** -150).all()


def check_product(a, a_scale, b, b_scale, bias, d):
    term = (a.double() @ b.double().t().contiguous()) * a_scale.double()[:, None] * b_scale.double()
    bias = torch.zeros(len(b), device="cuda", dtype=torch.float64) if bias is None else bias.double()
    off = 5 * 2.0 ** -24 * (term.abs() + bias.abs())
    over = (d.double() - term - bias).abs() - (2.0 ** -8 * ((term + bias).abs() + off) + off)
    assert (over <= 0).all(), over.max().item()


def relative(got, want):
    return ((got.double() - want.double()).norm() / want.double().norm()).item()


@pytest.mark.parametrize("tokens,hidden,wide", [(512, 1024, 4096), (1, 256, 512), (77, 512, 1040)])
def test_each_step_of_serving(example, tokens, hidden, wide):  # noqa: F811
    i = example.Inputs(tokens, hidden, wide, seed=tokens)
    s = example.Serving(i)
    for t in (s.h, s.y, s.a, s.q, s.out):
        t.fill_(3)
    s.run(i)
    torch.cuda.synchronize()
    for w, (q, scale) in ((i.up, s.up), (i.down, s.down)):
        check_codes(w, q, scale)
    test_block_norm.check(types.SimpleNamespace(
        x=i.x, z=i.z, r=i.r, weight=i.w, post_weight=i.pw, post=True, gate=True, branch=example.BRANCH, residual=1.0,
        y_type=INT8, h=s.h, y=s.y, scale=s.scale, rstd=s.rstd, post_rstd=s.post_rstd))
    check_product(s.y, s.scale, *s.up, i.bias, s.a)
    check_codes(s.a, s.q, s.a_scale)
    check_product(s.q, s.a_scale, *s.down, None, s.out)

    _, y = example.block(*(t.double() for t in (i.x, i.z, i.r, i.pw, i.w)))
    out = (y @ i.up.double().t().contiguous() + i.bias.double()) @ i.down.double().t().contiguous()
    parts = [relative(s.y.double() * s.scale.double()[:, None], y), relative(s.q.double() * s.a_scale.double()[:, None], s.a)]
    parts += [relative(q.double() * scale.double()[:, None], w) for w, (q, scale) in ((i.up, s.up), (i.down, s.down))]
    bound = 2 * sum(e * e for e in parts) ** 0.5 + 2.0 ** -7
    print("off by %.4f, allowed %.4f" % (relative(s.out, out), bound))
    assert bound < 0.1 and relative(s.out, out) <= bound
