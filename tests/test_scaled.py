"""The scaled 8-bit product against its definition in 64 bits.

Tolerance: the kernels add fp32 in the matrix instructions, over waves or
over K stages; the sum of K products is off by at most K * 2^-23 of the sum
of their magnitudes (the instructions may truncate rather than round: a whole
step, 2^-23, a product); the two scales add two roundings and the bf16 result
half a step, 2^-8."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED


def desc(M=5, N=7, K=100, a_rs=112, b_cs=112, d_rs=8, device=0, reserved=0):
    return migemm.migemm_scaled_desc(M, N, K, a_rs, b_cs, d_rs, device, reserved)


@pytest.mark.parametrize("over,status", [
    (dict(), OK),
    (dict(M=0), OK), (dict(N=0), OK), (dict(K=0), OK),
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD),
    (dict(reserved=2), BAD),
    (dict(a_rs=96), BAD), (dict(b_cs=96), BAD), (dict(d_rs=0), BAD),
    (dict(a_rs=104), MIS), (dict(b_cs=104), MIS), (dict(d_rs=12), MIS),
    (dict(a_rs=1 << 23), UNS), (dict(b_cs=1 << 23), UNS), (dict(d_rs=1 << 22), UNS),  # 256 rows: 2^31
    (dict(a_rs=(1 << 23) - 2048), OK),
    (dict(a_rs=1 << 62), UNS), (dict(M=1 << 62), UNS), (dict(N=1 << 62, d_rs=1 << 62), UNS),
])
def test_description_status(over, status):
    assert migemm.gemm_scaled_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_scaled_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_scaled_run(p, *[None] * 7) == BAD
        assert lib.gemm_scaled_workspace_size(p) == 0
    assert lib.gemm_scaled_plan_destroy(None) == OK
    assert lib.gemm_scaled_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_scaled_plan_create(None, None) == BAD


def storage(rows, cols, dtype, pad):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(per, -(-cols // per) * per) + pad * per
    full = torch.full((rows, ld), float("nan"), device="cuda").to(dtype)
    return full, full[:, :cols]


class Scaled:
    def __init__(self, M, N, K, pad=1, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K = M, N, K
        _, self.a = storage(M, K, torch.float8_e4m3fn, pad)
        _, self.b = storage(N, K, torch.float8_e4m3fn, pad)
        self.d_full, self.d = storage(M, N, torch.bfloat16, pad)
        self.a.copy_((torch.randn(M, K, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
        self.b.copy_((torch.randn(N, K, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
        self.sa = (torch.rand(M, generator=g) * 0.01 + 0.001).cuda()
        self.sb = (torch.rand(N, generator=g) * 0.01 + 0.001).cuda()
        self.plan = migemm.ScaledPlan(M, N, K, a_rs=self.a.stride(0), b_cs=self.b.stride(0),
                                      d_rs=self.d.stride(0))
        n = self.plan.workspace_size
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None

    def run(self, stream=None):
        self.plan.run(self.a, self.sa, self.b, self.sb, self.d, self.ws, stream)

    def check(self):
        a, b = self.a.cpu().float().double(), self.b.cpu().float().double()
        scale = self.sa.cpu().double()[:, None] * self.sb.cpu().double()
        want, size = (a @ b.t()) * scale, (a.abs() @ b.abs().t()) * scale
        got = self.d.cpu().double()
        assert torch.isfinite(got).all()
        bound = 2.0 ** -8 * want.abs() + (self.K + 4) * 2.0 ** -23 * size + 1e-38
        over = (got - want).abs() - bound
        assert (over <= 0).all(), (over.max().item(), over.argmax().item())
        assert torch.isnan(self.d_full[:, self.N:].float()).all()


# One row, few rows, every boundary of the small tiles and a step of K to
# either side; then sizes for the 256 x 256 tiles.
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 100, 127), (1, 8192, 8192), (3, 5, 129), (16, 16, 128),
          (17, 33, 300), (32, 32, 2048), (33, 31, 1000), (40, 1000, 4096), (48, 70, 4100),
          (49, 64, 96), (64, 200, 640), (65, 129, 513), (100, 64, 16384), (300, 500, 2000),
          (1, 3, 16), (7, 2000, 17), (130, 2, 8000), (1000, 1000, 1000), (2100, 4100, 700),
          (3000, 4000, 129), (257, 8200, 260)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    p = Scaled(M, N, K, seed=M + 3 * N + 7 * K)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
def test_scales_are_applied_to_their_row_and_column():
    p = Scaled(300, 300, 64, seed=4)
    p.a.fill_(1.0)
    p.b.fill_(1.0)
    p.sa.copy_(2.0 ** (torch.arange(300) % 7).float())
    p.sb.copy_(2.0 ** -(torch.arange(300) % 11).float())
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.d.float(), 64 * p.sa[:, None] * p.sb)   # exact in bf16


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 100), (40, 300), (2100, 4100)])
def test_a_nan_stays_in_its_row_and_column(M, N):
    p = Scaled(M, N, 200, seed=2)
    p.a[M // 2, 199] = float("nan")
    p.b[N // 3, 0] = float("nan")
    p.run()
    torch.cuda.synchronize()
    nan = torch.isnan(p.d.float()).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2, :] = True
    want[:, N // 3] = True
    assert torch.equal(nan, want)


@pytest.mark.gpu
def test_empty_products():
    for M, N, K in ((0, 5, 64), (5, 0, 64)):
        plan = migemm.ScaledPlan(M, N, K, a_rs=64, b_cs=64, d_rs=8)
        plan.run(None, None, None, None, None)
    for M, N in ((3, 40), (2100, 4100)):
        p = Scaled(M, N, 0)
        p.run()
        torch.cuda.synchronize()
        assert (p.d == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (40, 4096, 4096), (200, 500, 9000), (2100, 4100, 700)])
def test_runs_agree_on_streams_and_in_a_graph(M, N, K):
    p = Scaled(M, N, K, seed=6)
    p.run()
    torch.cuda.synchronize()
    want = p.d.clone()

    def same():
        torch.cuda.synchronize()
        ok = torch.equal(p.d, want)
        p.d.fill_(7)
        if p.ws is not None:
            p.ws.fill_(0xFF)
        torch.cuda.synchronize()
        return ok

    assert same()
    p.run(torch.cuda.Stream())
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(3):
        graph.replay()
        assert same()
        p.run()
        assert same()


@pytest.mark.gpu
def test_run_refusals():
    p = Scaled(4, 40, 64)
    lib, plan = migemm.load(), p.plan.handle
    a = [p.a.data_ptr(), p.sa.data_ptr(), p.b.data_ptr(), p.sb.data_ptr(), p.d.data_ptr()]
    for i in range(5):
        b = list(a)
        b[i] = None
        assert lib.gemm_scaled_run(plan, *b, None, None) == BAD
        b[i] = a[i] + 4
        assert lib.gemm_scaled_run(plan, *b, None, None) == MIS
    n = migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64)
    assert lib.gemm_scaled_run(n.handle, *a, None, None) == BAD
    handle = p.plan.handle
    assert lib.gemm_scaled_plan_destroy(handle) == OK
    p.plan.handle = None
    assert lib.gemm_scaled_run(handle, *a, None, None) == BAD
