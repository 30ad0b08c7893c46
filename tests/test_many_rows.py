"""More rows than a launch has workgroups for: a launch of the rows' quantization
and of the block norm's forward pass has at most 2^20, a checkpoint's at most
2^25 waves, and what is left takes further turns of the same workgroups.  What
the whole matrix gives is what its parts give, each in one turn, bit for bit."""
import pytest
import torch

from tests.test_operators_past_32_bits import need, normal
from warp_specialized_pipelined_amd import migemm

pytestmark = pytest.mark.gpu

BF16, E4M3, INT8 = migemm.MIGEMM_BF16, migemm.MIGEMM_FP8_E4M3, migemm.MIGEMM_INT8
BYTES = {BF16: 2, E4M3: 1, INT8: 1}
PART = 1 << 19


def up(v, to):
    return -(-v // to) * to


def matrix(rows, cols, size):
    """rows x cols elements of `size` bytes, as bytes, filled with 3."""
    return torch.full((rows, up(cols * size, 16)), 3, dtype=torch.uint8, device="cuda")


# Three turns: four rows a workgroup, and a row shared by four waves (whose sums
# alternate between two buffers).
SIZES = [((1 << 23) + 5, 7), ((1 << 21) + 5, 2056)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
def test_quantize(rows, cols, q_type):
    need(40)
    x = normal(rows, up(cols, 8))
    q, scale = matrix(rows, cols, 1), torch.full((rows,), 3.0, device="cuda")

    def plan(n):
        return migemm.QuantizePlan(n, cols, q_type, x_rs=x.stride(0), q_rs=q.stride(0))

    plan(rows).run(x, q, scale)
    part, part_scale = torch.empty_like(q[:PART]), torch.empty(PART, device="cuda")
    for first in range(0, rows, PART):
        n = min(PART, rows - first)
        some = plan(n) if n > 256 else plan(PART)  # (few rows would take another kernel)
        if n <= 256:
            first, n = rows - PART, PART
        part.fill_(3)
        some.run(x[first:], part, part_scale)
        torch.cuda.synchronize()
        assert torch.equal(q[first:first + n], part[:n]) and torch.equal(scale[first:first + n], part_scale[:n]), first


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("y_type,post,gate", [(INT8, True, False), (BF16, False, True)], ids=["int8", "bf16"])
def test_block_norm(rows, cols, y_type, post, gate):
    need(80)
    ld = up(cols, 8)
    x, r = normal(rows, ld), normal(rows, ld, 2.0)
    z = normal(rows, ld, 1.5) if gate else None
    w, pw = ((1 + 0.3 * torch.randn(cols, device="cuda")).bfloat16() for _ in range(2))

    def outputs(n):
        return [matrix(n, cols, 2), matrix(n, cols, BYTES[y_type])] + [
            torch.full((n,), 3.0, device="cuda") if used else None for used in (y_type != BF16, post, True)]

    def run(first, n, out):
        y_rs = out[1].stride(0) // BYTES[y_type]
        plan = migemm.BlockNormPlan(n, cols, 1e-5, y_type, x_rs=ld, r_rs=ld, h_rs=ld, y_rs=y_rs,
                                    z_rs=ld if gate else 0, post_norm=post)
        plan.run(x[first:], z[first:] if gate else None, r[first:], pw if post else None, w, *out)

    whole, part = outputs(rows), outputs(PART)
    run(0, rows, whole)
    for first in list(range(0, rows - PART, PART)) + [rows - PART]:
        for t in part:
            if t is not None:
                t.fill_(3)
        run(first, PART, part)
        torch.cuda.synchronize()
        for a, b in zip(whole, part):
            assert a is None or torch.equal(a[first:first + PART], b), first


def test_checkpoint():
    """One column, whose 32 tokens are a wave's work."""
    need(80)
    tokens, part = (1 << 30) + 103, 1 << 26
    x = torch.empty(tokens, 8, dtype=torch.bfloat16, device="cuda")
    for first in range(0, tokens, part):
        x[first:first + part] = torch.randn(min(part, tokens - first), 1, device="cuda").bfloat16()
    plan = migemm.CheckpointPlan(tokens, 1, x_rs=8)
    codes = plan.info.code_bytes
    assert codes == up(tokens, 32) * 16 and plan.checkpoint_size == codes * 33 // 32
    kept = torch.full((plan.checkpoint_size,), 3, dtype=torch.uint8, device="cuda")
    plan.pack(x, kept)
    back = torch.full((tokens, 8), 3.0, dtype=torch.bfloat16, device="cuda")
    plan.unpack(kept, back)
    torch.cuda.synchronize()
    for first in range(0, tokens, part):
        n = min(part, tokens - first)
        some = migemm.CheckpointPlan(n, 1, x_rs=8)
        k = torch.full((some.checkpoint_size,), 5, dtype=torch.uint8, device="cuda")
        some.pack(x[first:], k)
        b = torch.full((n, 8), 3.0, dtype=torch.bfloat16, device="cuda")
        some.unpack(k, b)
        torch.cuda.synchronize()
        c = some.info.code_bytes
        assert torch.equal(kept[first * 16:first * 16 + c], k[:c]), first
        assert torch.equal(kept[codes + first // 2:codes + first // 2 + c // 32], k[c:]), first
        assert torch.equal(back[first:first + n].view(torch.int16), b.view(torch.int16)), first
