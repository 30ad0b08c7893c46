"""The checkpoint's gradient where fp32 sums are exact: whole numbers of up to 15
(e4m3 holds them over their group's power) times whole numbers of up to 8, whose
sums over up to 131071 tokens stay below 2^24.  Then dw is the definition's, bit
for bit, whatever the order: a token that is lost or counted twice, a power of
another group, a sum that was rounded on its way between two launches all show.
Every kernel, whole and split, with an odd number of tokens."""
import pytest
import torch

from tests.test_block_kernels import KEPT
from tests.test_checkpoint import BF16, FP32, Checkpoint

pytestmark = pytest.mark.gpu


def run(tokens, cols, out_cols, dw_type, accumulate):
    g = torch.Generator(device="cuda").manual_seed(tokens + 5 * cols + 11 * out_cols)
    assert tokens * 15 * 8 < 1 << 24
    x = torch.randint(-15, 16, (tokens, cols), generator=g, device="cuda").bfloat16()
    # Powers of two that differ from column to column and from group to group.
    shift = torch.randint(-3, 1, (-(-tokens // 32), cols), generator=g, device="cuda").repeat_interleave(32, 0)[:tokens]
    x = torch.where(shift < -1, (x.float() / 4).round().bfloat16(), x)
    p = Checkpoint(tokens, cols, out_cols, dw_type, accumulate, x=x)
    p.dy.copy_(torch.randint(-8, 9, (tokens, out_cols), generator=g, device="cuda").bfloat16())
    p.x[tokens - 1] = 15       # the last token counts in every element
    p.dy[tokens - 1] = 8
    if accumulate:
        p.before = torch.randint(-1 << 20, 1 << 20, (out_cols, cols), generator=g, device="cuda").float()
        p.dw.copy_(p.before)
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    assert torch.equal(p.value().cuda(), p.x.double())     # nothing is lost in 8 bits
    want = p.dy.double().t().contiguous() @ p.x.double()
    if accumulate:
        want = want + p.before.double()
    assert want.abs().max() < 1 << 24
    # (bf16: the exact sum rounded once, which fp32 holds on its way.)
    assert torch.equal(p.dw, want.float().to(p.dw.dtype))
    assert torch.isnan(p.dw_full[:, p.cols:].float()).all()
    return p


@pytest.mark.parametrize("kernel,size", [(k, s) for k, sizes in KEPT for s in sizes])
@pytest.mark.parametrize("dw_type,accumulate", [(BF16, False), (FP32, False), (FP32, True)],
                         ids=["bf16", "fp32", "accumulate"])
def test_each_kernel(kernel, size, dw_type, accumulate):
    p = run(*size, dw_type, accumulate)
    i = p.plan.info
    if dw_type == BF16:
        assert (i.tile_m, i.tile_n, i.lds_stages, i.splits > 1) == kernel


@pytest.mark.parametrize("tokens", [1, 31, 32, 33, 63, 64, 65, 127, 129, 191, 193, 1025, 4097, 131071])
def test_each_end_of_the_tokens(tokens):
    run(tokens, 70, 90, FP32, False)


# Split over the tokens in fp32, too, with odd ends of each range.
@pytest.mark.parametrize("tokens,cols,out_cols", [(20001, 301, 203), (6725, 1001, 65), (13211, 8270, 490),
                                                  (10907, 6753, 147), (100003, 130, 60)])
@pytest.mark.parametrize("accumulate", [False, True], ids=["fp32", "accumulate"])
def test_split(tokens, cols, out_cols, accumulate):
    p = run(tokens, cols, out_cols, FP32, accumulate)
    assert p.plan.info.splits > 1
