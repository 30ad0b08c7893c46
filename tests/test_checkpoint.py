"""8-bit checkpoints and the weights' gradient from them, against their
definitions in 64 bits.

The kept form is the definition's, bit for bit: a bf16 value over a power of two
is exact in 64 bits, and so is its nearest code; what comes back is exact in
bf16.  The gradient: its products are exact; the sum of T of them in fp32 is off
by at most T 2^-23 of the sum of their magnitudes (a whole step each), and what
it is added to by one more; a bf16 result adds half a step, 2^-8."""
import ctypes

import pytest
import torch

from tests.test_quantize import e4m3_grid
from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED
BF16, FP32 = migemm.MIGEMM_BF16, migemm.MIGEMM_FP32


def desc(tokens=40, cols=100, x_rs=104, out_cols=30, dy_rs=32, dw_rs=104, dw_type=BF16, accumulate=0, device=0,
         reserved=0):
    return migemm.migemm_checkpoint_desc(tokens, cols, x_rs, out_cols, dy_rs, dw_rs, dw_type, accumulate, device,
                                         reserved)


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(tokens=0), OK), (dict(dw_type=FP32), OK), (dict(dw_type=FP32, accumulate=1), OK),
    (dict(out_cols=0, dy_rs=0, dw_rs=0), OK),                   # without a gradient
    (dict(tokens=-1), BAD), (dict(cols=0), BAD), (dict(out_cols=-1), BAD), (dict(reserved=1), BAD),
    (dict(out_cols=0), BAD), (dict(dy_rs=0), BAD), (dict(dw_rs=0), BAD),
    (dict(dw_type=2), BAD), (dict(dw_type=3), BAD), (dict(dw_type=0), BAD),
    (dict(accumulate=1), BAD), (dict(accumulate=2, dw_type=FP32), BAD),
    (dict(out_cols=0, dy_rs=0, dw_rs=0, dw_type=FP32, accumulate=1), BAD),
    (dict(x_rs=96), BAD), (dict(dy_rs=24), BAD), (dict(dw_rs=96), BAD),
    (dict(x_rs=100), MIS), (dict(dy_rs=36), MIS), (dict(dw_rs=100), MIS),
    (dict(dw_rs=100, dw_type=FP32), OK), (dict(dw_rs=102, dw_type=FP32), MIS),
    (dict(dy_rs=1 << 22), UNS), (dict(dw_rs=1 << 22), UNS), (dict(dw_rs=1 << 21, dw_type=FP32), UNS),
    (dict(tokens=(1 << 31) - 64), UNS), (dict(tokens=1 << 62), UNS), (dict(x_rs=1 << 61), UNS),
    (dict(cols=1 << 24, x_rs=1 << 24, dw_rs=1 << 24), UNS),
    (dict(cols=1 << 20, x_rs=1 << 20, dw_rs=1 << 20, out_cols=1 << 18, dy_rs=1 << 18), UNS),
    (dict(cols=1 << 20, x_rs=1 << 20, dw_rs=1 << 20, out_cols=(1 << 18) - 8, dy_rs=1 << 18), OK),
])
def test_description_status(over, status):
    assert migemm.gemm_checkpoint_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_checkpoint_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_checkpoint_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_checkpoint_pack(p, *[None] * 3) == BAD
        assert lib.gemm_checkpoint_unpack(p, *[None] * 3) == BAD
        assert lib.gemm_checkpoint_weight_gradient(p, *[None] * 5) == BAD
        assert lib.gemm_checkpoint_workspace_size(p) == 0
        assert lib.gemm_checkpoint_size(p) == 0
        assert lib.gemm_checkpoint_plan_get_info(p, ctypes.byref(info)) == BAD
    assert lib.gemm_checkpoint_plan_destroy(None) == OK
    assert lib.gemm_checkpoint_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_checkpoint_plan_create(None, None) == BAD
    assert lib.gemm_checkpoint_desc_validate(None) == BAD


def up(v, to):
    return -(-v // to) * to


def power(e):
    """2^e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def packed(x):
    """Codes (their values) and exponents, by the definition: NaN codes where x is not finite."""
    tokens, cols = x.shape
    v = torch.zeros(up(tokens, 32), up(cols, 16), dtype=torch.float64)
    v[:tokens, :cols] = x.cpu().double()
    v = v.view(-1, 32, v.shape[1])
    finite = torch.isfinite(v)
    top = torch.where(finite, v.abs(), 0.0).amax(1)
    e = torch.full(top.shape, 18)
    for p in range(18, 246):
        e += top > 448 * 2.0 ** (p - 127)
    codes = e4m3_grid(torch.where(finite, v, 0.0) / power(e - 127)[:, None])
    codes = torch.where(finite, codes, float("nan"))
    return codes, e


def strided(rows, cols, dtype, pad, fill=float("nan")):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    full = torch.full((rows, up(cols, per) + pad * per), fill, dtype=dtype, device="cuda")
    return full, full[:, :cols]


class Checkpoint:
    def __init__(self, tokens, cols, out_cols=0, dw_type=BF16, accumulate=False, pad=1, seed=0, x=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.cols, self.out_cols, self.accumulate = tokens, cols, out_cols, accumulate
        _, self.x = strided(tokens, cols, torch.bfloat16, pad)
        self.x.copy_(torch.randn(tokens, cols, generator=g, device="cuda") if x is None else x)
        kw = {}
        self.dw_type = dw_type
        if out_cols:
            _, self.dy = strided(tokens, out_cols, torch.bfloat16, pad)
            self.dy.copy_(torch.randn(tokens, out_cols, generator=g, device="cuda"))
            t = torch.float32 if dw_type == FP32 else torch.bfloat16
            self.dw_full, self.dw = strided(out_cols, cols, t, pad)
            self.before = None
            if accumulate:
                self.before = torch.randn(out_cols, cols, generator=g, device="cuda")
                self.dw.copy_(self.before)
            kw = dict(out_cols=out_cols, dy_rs=self.dy.stride(0), dw_rs=self.dw.stride(0), dw_type=dw_type,
                      accumulate=accumulate)
        self.plan = migemm.CheckpointPlan(tokens, cols, x_rs=self.x.stride(0), **kw)
        # 64 bytes of guard behind the kept form
        self.kept = torch.full((self.plan.checkpoint_size + 64,), 0x7E, dtype=torch.uint8, device="cuda")
        n = self.plan.workspace_size
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None

    def pack(self, stream=None):
        self.plan.pack(self.x, self.kept, stream)

    def gradient(self, stream=None):
        self.plan.weight_gradient(self.dy, self.kept, self.dw, self.ws, stream)

    def parts(self):
        tokens, ld = up(self.tokens, 32), up(self.cols, 16)
        i = self.plan.info
        assert (i.code_bytes, i.scale_bytes) == (tokens * ld, tokens * ld // 32)
        codes = self.kept[:tokens * ld].view(torch.float8_e4m3fn).float().double().cpu()
        codes = codes.view(-1, ld, 16).transpose(1, 2).reshape(-1, 32, ld)
        return codes, self.kept[tokens * ld:tokens * ld * 33 // 32].cpu().long().view(-1, ld)

    def value(self):
        """What is kept, tokens x cols, in 64 bits."""
        codes, e = self.parts()
        return (codes * power(e - 127)[:, None]).reshape(-1, codes.shape[2])[:self.tokens, :self.cols]

    def check_packed(self):
        codes, e = self.parts()
        want, exponents = packed(self.x)
        assert torch.equal(e, exponents)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(codes), nan)
        assert torch.equal(codes[~nan], want[~nan])
        assert (self.kept[self.plan.checkpoint_size:] == 0x7E).all()

    def check_gradient(self):
        kept, dy = self.value().cuda(), self.dy.double()
        want, size = dy.t().contiguous() @ kept, dy.abs().t().contiguous() @ kept.abs()
        if self.accumulate:
            want, size = want + self.before.double(), size + self.before.double().abs()
        got = self.dw.double()
        assert torch.isfinite(got).all()
        off = (self.tokens + 4) * 2.0 ** -23 * size
        if self.dw_type == BF16:
            off = off + 2.0 ** -8 * (want.abs() + off)
        over = (got - want).abs() - (off + 1e-38)
        assert (over <= 0).all(), (over.max().item(), over.argmax().item())
        assert torch.isnan(self.dw_full[:, self.cols:].float()).all()


PACKS = [(1, 1), (1, 8192), (31, 7), (32, 16), (33, 17), (64, 255), (65, 256), (500, 257), (1001, 300), (7, 1031)]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols", PACKS)
def test_pack_and_unpack(tokens, cols):
    p = Checkpoint(tokens, cols, seed=tokens + cols)
    p.pack()
    torch.cuda.synchronize()
    p.check_packed()
    full, back = strided(tokens, cols, torch.bfloat16, 1)
    plan = migemm.CheckpointPlan(tokens, cols, x_rs=back.stride(0))
    plan.unpack(p.kept, back)
    torch.cuda.synchronize()
    assert torch.equal(back.double().cpu(), p.value())
    assert torch.isnan(full[:, cols:].float()).all()


@pytest.mark.gpu
def test_pack_of_every_magnitude():
    """Groups over the whole range of bf16: random patterns of a binade or of
    eight below a largest one, of each exponent."""
    g = torch.Generator().manual_seed(5)
    exponents = torch.arange(0, 255).repeat_interleave(24)
    cols = len(exponents)
    below = torch.tensor([1, 2, 9, 20])[torch.arange(cols) % 4]
    e = (exponents - (torch.rand(32, cols, generator=g) * below).long()).clamp(min=0)
    bits = (e << 7) | torch.randint(0, 128, (32, cols), generator=g)
    bits |= torch.randint(0, 2, (32, cols), generator=g) << 15
    x = torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(torch.bfloat16)
    p = Checkpoint(32, cols, x=x)
    assert torch.equal(p.x.cpu().view(torch.int16), x.view(torch.int16))
    p.pack()
    back = torch.empty_like(p.x)
    plan = migemm.CheckpointPlan(32, cols, x_rs=up(cols, 8))
    full, back = strided(32, cols, torch.bfloat16, 0)
    plan.unpack(p.kept, back)
    torch.cuda.synchronize()
    p.check_packed()
    assert torch.equal(back.double().cpu(), p.value())


@pytest.mark.gpu
def test_pack_of_zeros_nan_and_infinity():
    p = Checkpoint(70, 40, seed=3)
    p.x[:, 0] = 0
    p.x[5, 1] = float("nan")
    p.x[40, 2] = float("inf")
    p.x[69, 3] = float("-inf")
    p.x[:, 4] = float("nan")
    p.x[3, 5] = 3.3895e38                                # past 1.75 * 2^127
    p.x[4, 5] = float("nan")
    p.x[:, 6] = 2.0 ** -130
    p.pack()
    torch.cuda.synchronize()
    p.check_packed()
    full, back = strided(70, 40, torch.bfloat16, 1)
    p.plan.unpack(p.kept, back)
    torch.cuda.synchronize()
    back, value = back.double().cpu(), p.value()
    assert torch.equal(torch.isnan(back), torch.isnan(value))
    assert torch.equal(back[~torch.isnan(back)], value[~torch.isnan(value)])


# Tokens to either side of a group and of a stage, columns to either side of the
# tiles; one token; one row of the gradient.
GRADIENTS = [(1, 1, 1), (1, 300, 70), (16, 64, 64), (31, 33, 65), (32, 65, 33), (33, 128, 129), (63, 16, 500),
             (64, 129, 128), (65, 200, 300), (100, 255, 257), (128, 257, 255), (257, 100, 1000), (1001, 300, 200),
             (4096, 64, 64), (5000, 70, 130), (300, 1, 2000), (300, 2000, 1), (1000, 1100, 1300), (700, 2100, 4100)]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols,out_cols", GRADIENTS)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "accumulate"])
def test_weight_gradient(tokens, cols, out_cols, kind):
    p = Checkpoint(tokens, cols, out_cols, BF16 if kind == "bf16" else FP32, kind == "accumulate",
                   seed=tokens + 3 * cols + 7 * out_cols)
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    p.check_gradient()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols,out_cols", [(50, 100, 90), (3000, 600, 520)])
def test_a_nan_stays_in_its_row_and_column(tokens, cols, out_cols):
    """dy's NaN in its row of dw, x's in its column; and what lies beside the
    operands (strided() fills it with NaN) in neither."""
    p = Checkpoint(tokens, cols, out_cols, seed=8)
    p.x[tokens - 1, cols // 3] = float("nan")
    p.dy[tokens - 2, out_cols // 2] = float("nan")
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    want = torch.zeros(out_cols, cols, dtype=torch.bool, device="cuda")
    want[:, cols // 3] = True
    want[out_cols // 2] = True
    assert torch.equal(torch.isnan(p.dw.float()), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dw_type,accumulate", [(BF16, False), (FP32, False), (FP32, True)])
def test_no_tokens(dw_type, accumulate):
    p = Checkpoint(0, 100, 300, dw_type, accumulate)
    assert p.plan.checkpoint_size == 0
    p.pack()
    p.plan.unpack(p.kept, p.x)
    p.gradient()
    torch.cuda.synchronize()
    assert torch.equal(p.dw, p.before if accumulate else torch.zeros_like(p.dw))


@pytest.mark.gpu
def test_gradient_against_differences():
    """<dw, v> is the change of F(W) = sum dy (x~ W^T) along v: F is linear, so
    one difference gives it, in 64 bits."""
    p = Checkpoint(200, 90, 70, FP32, seed=4)
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    kept, dy = p.value(), p.dy.cpu().double()
    g = torch.Generator().manual_seed(2)
    w = torch.randn(70, 90, generator=g, dtype=torch.float64)
    size = dy.abs().t() @ kept.abs()
    for _ in range(4):
        v = torch.randn(70, 90, generator=g, dtype=torch.float64)
        diff = ((dy * (kept @ (w + v).t())).sum() - (dy * (kept @ (w - v).t())).sum()) / 2
        got = (p.dw.cpu().double() * v).sum()
        assert abs(got - diff) <= 204 * 2.0 ** -23 * (size * v.abs()).sum() + 1e-9


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,cols,out_cols", [(600, 300, 200), (8192, 200, 300), (1000, 2100, 4100)])
def test_runs_agree_on_streams_and_in_a_graph(tokens, cols, out_cols):
    p = Checkpoint(tokens, cols, out_cols, FP32, seed=9)
    p.pack()
    p.gradient()
    torch.cuda.synchronize()
    want = [p.kept.clone(), p.dw.clone()]

    def same():
        torch.cuda.synchronize()
        return torch.equal(p.kept, want[0]) and torch.equal(p.dw, want[1])

    def spoil():
        p.kept[:p.plan.checkpoint_size] = 3
        p.dw.fill_(7)
        if p.ws is not None:
            p.ws.fill_(0xFF)
        torch.cuda.synchronize()

    spoil()
    s = torch.cuda.Stream()
    p.pack(s)
    p.gradient(s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.pack()
        p.gradient()
    for _ in range(3):
        spoil()
        graph.replay()
        assert same()
        p.pack()
        p.gradient()
        assert same()


@pytest.mark.gpu
def test_run_refusals():
    p = Checkpoint(40, 100, 30)
    lib, plan = migemm.load(), p.plan.handle
    x, kept, dy, dw = (t.data_ptr() for t in (p.x, p.kept, p.dy, p.dw))
    for f, args in ((lib.gemm_checkpoint_pack, [x, kept]), (lib.gemm_checkpoint_unpack, [kept, x])):
        for i in range(2):
            b = list(args)
            b[i] = None
            assert f(plan, *b, None) == BAD
            b[i] = args[i] + 4
            assert f(plan, *b, None) == MIS
    args = [dy, kept, dw]
    for i in range(3):
        b = list(args)
        b[i] = None
        assert lib.gemm_checkpoint_weight_gradient(plan, *b, None, None) == BAD
        b[i] = args[i] + 4
        assert lib.gemm_checkpoint_weight_gradient(plan, *b, None, None) == MIS
    q = migemm.CheckpointPlan(40, 100, x_rs=104)                         # no gradient
    assert q.workspace_size == 0
    assert lib.gemm_checkpoint_weight_gradient(q.handle, *args, None, None) == BAD
    n = migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64)
    assert lib.gemm_checkpoint_pack(n.handle, x, kept, None) == BAD      # another kind of plan
