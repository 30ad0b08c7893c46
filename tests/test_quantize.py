"""Rows to 8 bits against the definition in 64 bits.

The codes are the definition's, every one: x and max |x| have 8 significant
bits, so that x top / max |x| is either on the border of two codes, where 64 bits
hold it exactly, or 2^-17 of itself away from one.  The scale is one division in
fp32: half a step, 2^-24 (or 2^-150 among subnormals)."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED
INT8, E4M3 = migemm.MIGEMM_INT8, migemm.MIGEMM_FP8_E4M3
TOP = {INT8: 127.0, E4M3: 448.0}
TYPE = {INT8: torch.int8, E4M3: torch.float8_e4m3fn}


def desc(rows=4, cols=100, x_rs=104, q_rs=112, q_type=INT8, device=0, reserved=0):
    return migemm.migemm_quantize_desc(rows, cols, x_rs, q_rs, q_type, device, reserved)


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(q_type=E4M3), OK), (dict(rows=0), OK),
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(reserved=1), BAD),
    (dict(q_type=1), BAD), (dict(q_type=4), BAD), (dict(q_type=0), BAD),
    (dict(x_rs=96), BAD), (dict(q_rs=96), BAD), (dict(x_rs=100), MIS), (dict(q_rs=104), MIS),
    (dict(cols=32768, x_rs=32768, q_rs=32768), OK), (dict(cols=32769, x_rs=32776, q_rs=32784), UNS),
    (dict(rows=1 << 62), UNS), (dict(x_rs=1 << 61), UNS),
])
def test_description_status(over, status):
    assert migemm.gemm_quantize_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_quantize_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_quantize_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_quantize_run(p, *[None] * 4) == BAD
        assert lib.gemm_quantize_workspace_size(p) == 0
        assert lib.gemm_quantize_plan_get_info(p, ctypes.byref(info)) == BAD
    assert lib.gemm_quantize_plan_destroy(None) == OK
    assert lib.gemm_quantize_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_quantize_plan_create(None, None) == BAD
    assert lib.gemm_quantize_desc_validate(None) == BAD


def e4m3_grid(v):
    """The nearest e4m3 values, ties to even."""
    _, e = torch.frexp(v)
    step = (((e.to(torch.int64) - 1).clamp(min=-6) - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(v / step) * step).clamp(-448, 448)


class Rows:
    def __init__(self, x, q_type=INT8, pad=1):
        self.rows, self.cols = x.shape
        ld = -(-self.cols // 8) * 8 + 8 * pad
        full = torch.full((self.rows, ld), float("nan"), device="cuda").bfloat16()
        self.x = full[:, :self.cols]
        self.x.copy_(x)
        ld = -(-self.cols // 16) * 16 + 16 * pad
        self.q_full = torch.full((self.rows, ld), 5, dtype=torch.int8, device="cuda")
        self.q = self.q_full.view(TYPE[q_type])[:, :self.cols]
        self.scale = torch.full((self.rows,), 7.0, device="cuda")
        self.q_type = q_type
        self.plan = migemm.QuantizePlan(self.rows, self.cols, q_type, x_rs=self.x.stride(0), q_rs=self.q.stride(0))

    def run(self, stream=None):
        self.plan.run(self.x, self.q, self.scale, stream)

    def check(self):
        x = self.x.double()
        largest = x.abs().amax(1)
        v = x * TOP[self.q_type] / torch.where(largest > 0, largest, 1.0)[:, None]
        want = torch.round(v) if self.q_type == INT8 else e4m3_grid(v)
        assert torch.equal(self.q.float().double(), want)
        scale = largest / TOP[self.q_type]
        assert ((self.scale.double() - scale).abs() <= 2.0 ** -24 * scale + 2.0 ** -150).all()
        assert (self.q_full[:, self.cols:] == 5).all()


SHAPES = [(1, 1), (1, 8192), (3, 7), (5, 64), (300, 511), (37, 512), (9, 513), (70, 1024), (6, 1031),
          (129, 2048), (4, 2049), (33, 5000), (1030, 300), (2, 8193), (3, 32768), (600, 4096), (300, 16385)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
def test_rows(rows, cols, q_type):
    g = torch.Generator().manual_seed(rows * 5 + cols)
    p = Rows(torch.randn(rows, cols, generator=g).bfloat16(), q_type)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
def test_every_pair_of_a_significand_and_a_largest_one(q_type):
    """Rows whose largest magnitude has each of the 128 significands, at small,
    ordinary and large powers; in each every smaller value of 14 binades: all
    the quotients there are, those on the borders of codes among them."""
    bits = torch.arange(0, 14 * 128, dtype=torch.int32)
    values = ((bits + ((127 - 13) << 7)).to(torch.int16)).view(torch.bfloat16).double()   # 2^-13 .. < 2
    rows = []
    for power in (-112, -80, -63, -62, -61, 0, 63, 64, 65, 120, 126):
        for m in range(128):
            largest = 1 + m / 128
            row = torch.where(values <= largest, values, values / 2)
            row[1::2] *= -1
            row = torch.cat([row, torch.tensor([largest], dtype=torch.float64)])
            rows.append(row * 2.0 ** power)
    p = Rows(torch.stack(rows).bfloat16(), q_type)
    assert torch.equal(p.x.double().cpu(), torch.stack(rows))
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("q_type", [INT8, E4M3], ids=["int8", "e4m3"])
def test_rows_of_zeros_subnormals_nan_and_infinity(q_type):
    x = torch.randn(6, 600, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[1] = 0
    x[2, 599] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = 2.0 ** -133                                   # the smallest subnormal
    x[4, 7] = 0
    x[5] = 3.3895e38                                     # the largest finite value
    p = Rows(x, q_type)
    p.run()
    torch.cuda.synchronize()
    q, scale = p.q.float().cpu(), p.scale.cpu()
    assert scale[1] == 0 and (q[1] == 0).all()
    assert torch.isnan(scale[2:4]).all() and (q[2:4] == 0).all()
    assert (q[4] == torch.where(torch.arange(600) == 7, 0.0, TOP[q_type])).all()
    assert (q[5] == TOP[q_type]).all() and torch.isfinite(scale[5])
    assert abs(scale[4].item() - 2.0 ** -133 / TOP[q_type]) <= 2.0 ** -150


@pytest.mark.gpu
def test_no_rows():
    plan = migemm.QuantizePlan(0, 100, x_rs=104, q_rs=112)
    plan.run(None, None, None)


@pytest.mark.gpu
def test_kernels_and_runs_on_streams_and_in_a_graph():
    for rows, cols, shape in ((1, 512, (1, 1)), (2000, 1000, (1, 2)), (2000, 2000, (1, 4)), (5, 2048, (4, 1)),
                              (300, 4000, (4, 2)), (300, 8192, (4, 4)), (3, 8000, (16, 1)), (3, 16000, (16, 2)),
                              (3, 32000, (16, 4))):
        p = Rows(torch.randn(rows, cols, generator=torch.Generator().manual_seed(3)).bfloat16())
        assert (p.plan.info.waves, p.plan.info.vectors) == shape
        p.run()
        torch.cuda.synchronize()
        p.check()
        q, scale = p.q.clone(), p.scale.clone()
        p.run(torch.cuda.Stream())
        torch.cuda.synchronize()
        assert torch.equal(p.q, q) and torch.equal(p.scale, scale)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.run()
        for _ in range(3):
            p.q.fill_(3)
            p.scale.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(p.q, q) and torch.equal(p.scale, scale)


@pytest.mark.gpu
def test_run_refusals():
    p = Rows(torch.ones(4, 100))
    lib, plan = migemm.load(), p.plan.handle
    a = [p.x.data_ptr(), p.q.data_ptr(), p.scale.data_ptr()]
    for i in range(3):
        b = list(a)
        b[i] = None
        assert lib.gemm_quantize_run(plan, *b, None) == BAD
        b[i] = a[i] + 2
        assert lib.gemm_quantize_run(plan, *b, None) == MIS
    n = migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64)
    assert lib.gemm_quantize_run(n.handle, *a, None) == BAD          # another kind of plan
