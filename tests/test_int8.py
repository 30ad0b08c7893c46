"""The int8 product against its definition in 64 bits.

Tolerance: the sum is exact in int32; its conversion to fp32, the two scales and
the bias's addition round by half a step each, 2^-24 of what they give (four of
them, of at most |sum a_scale b_scale| + |bias|; 5 for the terms of second
order), the bf16 result by 2^-8."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED


def desc(M=5, N=7, K=100, a_rs=112, b_cs=112, d_rs=8, device=0, reserved=0):
    return migemm.migemm_int8_desc(M, N, K, a_rs, b_cs, d_rs, device, reserved)


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
    (dict(K=131071, a_rs=131072, b_cs=131072), OK),
    (dict(K=131072, a_rs=131072, b_cs=131072), UNS),      # 131072 * 128 * 128 = 2^31
])
def test_description_status(over, status):
    assert migemm.gemm_int8_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_an_int8_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_int8_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_int8_run(p, *[None] * 8) == BAD
        assert lib.gemm_int8_workspace_size(p) == 0
        assert lib.gemm_int8_plan_get_info(p, ctypes.byref(info)) == BAD
    assert lib.gemm_int8_plan_destroy(None) == OK
    assert lib.gemm_int8_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_int8_plan_create(None, None) == BAD
    assert lib.gemm_int8_desc_validate(None) == BAD


def storage(rows, cols, dtype, pad, fill):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = max(per, -(-cols // per) * per) + pad * per
    full = torch.full((rows, ld), fill, dtype=dtype, device="cuda")
    return full, full[:, :cols]


class Int8:
    def __init__(self, M, N, K, pad=1, seed=0, bias=True, low=-128):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K = M, N, K
        # What lies past a row's columns is poison: codes that would change every sum.
        _, self.a = storage(M, K, torch.int8, pad, 101)
        _, self.b = storage(N, K, torch.int8, pad, -77)
        self.d_full, self.d = storage(M, N, torch.bfloat16, pad, float("nan"))
        self.a.copy_(torch.randint(low, 128, (M, K), generator=g, dtype=torch.int8))
        self.b.copy_(torch.randint(low, 128, (N, K), generator=g, dtype=torch.int8))
        self.sa = (torch.rand(M, generator=g) * 0.01 + 0.001).cuda()
        self.sb = (torch.rand(N, generator=g) * 0.01 + 0.001).cuda()
        self.bias = torch.randn(N, generator=g).cuda() if bias else None
        self.plan = migemm.Int8Plan(M, N, K, a_rs=self.a.stride(0), b_cs=self.b.stride(0), d_rs=self.d.stride(0))
        n = self.plan.workspace_size
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None

    def run(self, stream=None):
        self.plan.run(self.a, self.sa, self.b, self.sb, self.bias, self.d, self.ws, stream)

    def check(self):
        # (Sums below 2^53: exact in 64 bits.)
        term = (self.a.double() @ self.b.double().t()) * self.sa.double()[:, None] * self.sb.double()
        bias = self.bias.double() if self.bias is not None else torch.zeros((), dtype=torch.float64, device="cuda")
        want = term + bias
        got = self.d.double()
        assert torch.isfinite(got).all()
        off = 5 * 2.0 ** -24 * (term.abs() + bias.abs())
        over = (got - want).abs() - (2.0 ** -8 * (want.abs() + off) + off + 1e-38)
        assert (over <= 0).all(), (over.max().item(), over.argmax().item())
        assert torch.isnan(self.d_full[:, self.N:].float()).all()


# One row, few rows, every boundary of the small tiles and a step of K to
# either side; then sizes for the large tiles.
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 100, 127), (1, 8192, 8192), (3, 5, 129), (16, 16, 128),
          (17, 33, 300), (32, 32, 2048), (33, 31, 1000), (40, 1000, 4096), (48, 70, 4100),
          (49, 64, 96), (64, 200, 640), (65, 129, 513), (100, 64, 16384), (300, 500, 2000),
          (1, 3, 16), (7, 2000, 17), (130, 2, 8000), (1000, 1000, 1000), (2100, 4100, 700),
          (3000, 4000, 129), (257, 8200, 260)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bias", [True, False], ids=["bias", "plain"])
def test_product(M, N, K, bias):
    p = Int8(M, N, K, seed=M + 3 * N + 7 * K, bias=bias)
    p.run()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 40), (60, 200), (300, 300)])
def test_the_largest_sums(M, N):
    """-128 times -128, at the longest K: 131071 * 2^14 < 2^31, which fp32 holds exactly."""
    p = Int8(M, N, 131071, bias=False)
    p.a.fill_(-128)
    p.b.fill_(-128)
    p.sa.fill_(2.0 ** -10)
    p.sb.fill_(2.0 ** -20)
    p.b[N - 1] = 127                                       # and the most negative ones
    p.run()
    torch.cuda.synchronize()
    p.check()
    assert (p.d[:, 0].float() == 2.0).all()                # (2^31 - 2^14) 2^-30, rounded


@pytest.mark.gpu
def test_scales_and_bias_are_applied_to_their_row_and_column():
    p = Int8(300, 300, 64, seed=4)
    p.a.fill_(1)
    p.b.fill_(1)
    p.sa.copy_(2.0 ** (torch.arange(300) % 3).float())
    p.sb.copy_(2.0 ** -(torch.arange(300) % 3).float())
    p.bias.copy_((torch.arange(300) % 8).float() * 4)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.d.float(), 64 * p.sa[:, None] * p.sb + p.bias)   # multiples of 4 up to 284... exact
    p.bias = None
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.d.float(), 64 * p.sa[:, None] * p.sb)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 100), (40, 300), (2100, 4100)])
def test_a_nan_scale_stays_in_its_row_and_column(M, N):
    p = Int8(M, N, 200, seed=2)
    p.sa[M // 2] = float("nan")
    p.sb[N // 3] = float("inf")
    p.bias[N // 2] = float("nan")
    p.b[N // 3] = 0                                        # 0 * infinity
    p.run()
    torch.cuda.synchronize()
    nan = torch.isnan(p.d.float()).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[M // 2, :] = True
    want[:, N // 3] = True
    want[:, N // 2] = True
    assert torch.equal(nan, want)


@pytest.mark.gpu
def test_empty_products():
    for M, N, K in ((0, 5, 64), (5, 0, 64)):
        plan = migemm.Int8Plan(M, N, K, a_rs=64, b_cs=64, d_rs=8)
        plan.run(None, None, None, None, None, None)
    for M, N in ((3, 40), (2100, 4100)):
        p = Int8(M, N, 0)
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(p.d, p.bias.bfloat16().expand(M, N))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (40, 4096, 4096), (200, 500, 9000), (2100, 4100, 700)])
def test_runs_agree_on_streams_and_in_a_graph(M, N, K):
    p = Int8(M, N, K, seed=6)
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
    p = Int8(4, 40, 64)
    lib, plan = migemm.load(), p.plan.handle
    a = [p.a.data_ptr(), p.sa.data_ptr(), p.b.data_ptr(), p.sb.data_ptr(), p.bias.data_ptr(), p.d.data_ptr()]
    for i in range(6):
        b = list(a)
        if i != 4:
            b[i] = None
            assert lib.gemm_int8_run(plan, *b, None, None) == BAD
        b[i] = a[i] + 4
        assert lib.gemm_int8_run(plan, *b, None, None) == MIS
    n = migemm.ScaledPlan(4, 40, 64, a_rs=64, b_cs=64, d_rs=40)
    assert lib.gemm_int8_run(n.handle, *a, None, None) == BAD          # another kind of plan
    handle = p.plan.handle
    assert lib.gemm_int8_plan_destroy(handle) == OK
    p.plan.handle = None
    assert lib.gemm_int8_run(handle, *a, None, None) == BAD
