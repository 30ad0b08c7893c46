"""The norm operator against its definition in 64 bits: forward in bf16 and
e4m3, gradients, refusals.

Tolerances.  Sums run over at most 32 values a lane, then a tree over 64
lanes and up to 16 waves: fewer than 64 roundings, so a sum of positive terms
is off by at most 64 * 2^-24 of itself, and rstd by half of that and 2 units
of its own; SUM = 80 * 2^-24 covers both.  A bf16 output adds half a step,
2^-8 of the value, an e4m3 code 2^-4 of it (or 2^-10 among subnormals)."""
import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED
BF16, E4M3 = migemm.MIGEMM_BF16, migemm.MIGEMM_FP8_E4M3
SUM = 80 * 2.0 ** -24
EPS = 1e-5


def desc(rows=4, cols=100, x_rs=104, y_rs=104, r_rs=104, h_rs=104, dy_rs=104, dx_rs=104, dh_rs=104,
         eps=EPS, y_type=BF16, device=0, reserved=0):
    return migemm.migemm_norm_desc(rows, cols, x_rs, y_rs, r_rs, h_rs, dy_rs, dx_rs, dh_rs, eps,
                                   y_type, device, reserved)


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("over,status", [
    (dict(), OK),
    (dict(rows=0), OK),
    (dict(rows=-1), BAD),
    (dict(cols=0), BAD),
    (dict(cols=-3), BAD),
    (dict(x_rs=96), BAD),                                  # shorter than the columns
    (dict(x_rs=100), MIS),                                 # 200-byte rows
    (dict(y_rs=100), MIS),
    (dict(y_type=E4M3, y_rs=104), MIS),                    # 104-byte rows of codes
    (dict(y_type=E4M3, y_rs=112), OK),
    (dict(y_type=3), BAD),
    (dict(eps=0.0), BAD),
    (dict(eps=-1e-5), BAD),
    (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD),
    (dict(r_rs=0), BAD),                                   # a residual out without one in
    (dict(h_rs=0), BAD),
    (dict(r_rs=0, h_rs=0), OK),
    (dict(dy_rs=0), BAD),
    (dict(dx_rs=0), BAD),
    (dict(dy_rs=0, dx_rs=0), BAD),                         # dh without a backward pass
    (dict(dy_rs=0, dx_rs=0, dh_rs=0), OK),
    (dict(dh_rs=0), OK),
    (dict(reserved=1), BAD),
    (dict(cols=32769, **{k: 32776 for k in ("x_rs", "y_rs", "r_rs", "h_rs", "dy_rs", "dx_rs", "dh_rs")}),
     UNS),
    (dict(cols=32768, **{k: 32768 for k in ("x_rs", "y_rs", "r_rs", "h_rs", "dy_rs", "dx_rs", "dh_rs")}),
     OK),
    (dict(x_rs=1 << 61), UNS),
    (dict(rows=1 << 62), UNS),
])
def test_description_status(over, status):
    assert migemm.gemm_norm_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_norm_plan():
    import ctypes
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_norm_run(p, *[None] * 8) == BAD
        assert lib.gemm_norm_run_backward(p, *[None] * 9) == BAD
        assert lib.gemm_norm_workspace_size(p) == 0
    assert lib.gemm_norm_plan_destroy(None) == OK
    assert lib.gemm_norm_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_norm_plan_create(None, None) == BAD
    assert junk.raw == b"\xff" * 4096 + b"\x00"


# ---------------------------------------------------------------- GPU plumbing

def strided(rows, cols, dtype, pad, fill="nan"):
    """A rows x cols view whose rows start on 16 bytes; the rest is poisoned."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = -(-cols // per) * per + pad * per
    full = torch.full((rows, ld), float(fill), device="cuda").to(dtype)
    return full, full[:, :cols]


class Norm:
    def __init__(self, rows, cols, y_type=BF16, residual=True, pad=1, seed=0, spread=1.0, shift=None):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.cols, self.y_type, self.residual = rows, cols, y_type, residual

        def filled(scale):
            full, v = strided(rows, cols, torch.bfloat16, pad)
            v.copy_((torch.randn(rows, cols, generator=g) * scale).bfloat16())
            return v

        self.x, self.r = filled(spread), filled(2 * spread)
        self.dy, self.dh = filled(0.5), filled(0.25)
        self.weight = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16().cuda()
        self.fulls = {}
        for name, t in (("y", torch.float8_e4m3fn if y_type == E4M3 else torch.bfloat16),
                        ("h", torch.bfloat16), ("dx", torch.bfloat16)):
            full, v = strided(rows, cols, t, pad)
            self.fulls[name] = full
            setattr(self, name, v)
        self.rstd = torch.full((rows,), float("nan"), device="cuda")
        self.scale = torch.full((rows,), float("nan"), device="cuda") if y_type == E4M3 else None
        self.dweight = torch.full((cols,), float("nan"), device="cuda")
        rs = {k: getattr(self, k[:-3]).stride(0) for k in ("x_rs", "y_rs", "dy_rs", "dx_rs")}
        if residual:
            rs.update(r_rs=self.r.stride(0), h_rs=self.h.stride(0), dh_rs=self.dh.stride(0))
        self.plan = migemm.NormPlan(rows, cols, EPS, y_type, **rs)
        self.ws = torch.full((self.plan.workspace_size,), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        self.plan.run(self.x, self.r if self.residual else None, self.weight,
                      self.h if self.residual else None, self.y, self.scale, self.rstd, stream)

    def backward(self, stream=None):
        self.plan.run_backward(self.dy, self.h if self.residual else self.x, self.weight, self.rstd,
                               self.dh if self.residual else None, self.dx, self.dweight, self.ws, stream)

    def reference(self):
        x = self.x.cpu().double()
        h = (x + self.r.cpu().double()).bfloat16().double() if self.residual else x
        w = self.weight.cpu().double()
        rstd = (h.pow(2).mean(1) + EPS).rsqrt()
        n = h * rstd[:, None]
        g = self.dy.cpu().double()
        gwn = g * w * n
        d = rstd[:, None] * (g * w - n * gwn.mean(1, keepdim=True))
        size = rstd[:, None].abs() * ((g * w).abs() + n.abs() * gwn.abs().mean(1, keepdim=True))
        if self.residual:
            d, size = d + self.dh.cpu().double(), size + self.dh.cpu().double().abs()
        return dict(h=h, rstd=rstd, y=n * w, dx=d, dx_size=size, dweight=(g * n).sum(0),
                    dweight_size=(g * n).abs().sum(0))


def within(got, want, bound):
    got = got.cpu().double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (over.max().item(), over.argmax().item())


def check(p):
    ref = p.reference()
    if p.residual:
        assert torch.equal(p.h.cpu().double(), ref["h"])
    within(p.rstd, ref["rstd"], SUM * ref["rstd"])
    y = ref["y"]
    if p.y_type == BF16:
        within(p.y, y, (2.0 ** -8 + SUM) * y.abs() + 1e-38)
    else:
        scale = y.abs().amax(1) / 448
        within(p.scale, scale, SUM * scale + 1e-44)
        q = torch.where(scale[:, None] > 0, y / scale[:, None], 0.0)
        step = torch.maximum(2.0 ** -4 * q.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64))
        within(p.y.float(), q, step * (1 + 2.0 ** -16) + SUM * q.abs())
        top = y.abs().amax(1) > 0
        assert (p.y.float().abs().amax(1).cpu()[top] == 448).all()


def check_backward(p):
    ref = p.reference()
    # dx: the mean's and the products' roundings are within SUM of the terms' sizes
    within(p.dx, ref["dx"], 2.0 ** -8 * ref["dx"].abs() + 2 * SUM * ref["dx_size"] + 1e-38)
    # dweight: rows / walkers additions a walker, then 48 over the partial rows
    within(p.dweight, ref["dweight"], (p.rows / 512 + 100) * 2.0 ** -24 * ref["dweight_size"])


def untouched(p, names):
    for n in names:
        full = p.fulls[n][:, p.cols:]
        assert torch.isnan(full.float()).all(), n


SHAPES = [(1, 1), (1, 8192), (3, 7), (5, 64), (300, 511), (37, 512), (9, 513), (70, 1024), (6, 1031),
          (129, 2048), (4, 2049), (33, 5000), (1030, 300), (2, 8193), (3, 32768), (600, 4096)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("y_type", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("residual", [True, False], ids=["residual", "plain"])
def test_forward_and_gradients(rows, cols, y_type, residual):
    p = Norm(rows, cols, y_type, residual, seed=rows * 7 + cols)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p)
    check_backward(p)
    untouched(p, ["y", "dx"] + (["h"] if residual else []))


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-18, 1e-3, 1e4, 1e15])
@pytest.mark.parametrize("y_type", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_magnitudes(spread, y_type):
    p = Norm(20, 777, y_type, seed=5, spread=spread)
    p.forward()
    torch.cuda.synchronize()
    check(p)


@pytest.mark.gpu
def test_rows_of_zeros_nan_and_infinity():
    for y_type in (BF16, E4M3):
        p = Norm(6, 600, y_type, residual=False, seed=1)
        p.x[1] = 0
        p.x[2, 599] = float("nan")
        p.x[3, 0] = float("inf")
        p.x[4] = 1e-40        # bf16 subnormals
        p.forward()
        torch.cuda.synchronize()
        y = p.y.float().cpu()
        assert (y[1] == 0).all()
        assert torch.isnan(y[2]).all()
        assert torch.isnan(y[3, 0]) and (y[3, 1:] == 0).all()
        assert torch.isfinite(y[[0, 1, 4, 5]]).all()
        if y_type == E4M3:
            scale = p.scale.cpu()
            assert scale[1] == 0 and torch.isnan(scale[2]) and torch.isnan(scale[3])
            assert scale[4] > 0 and y[4].abs().max() == 448


@pytest.mark.gpu
def test_no_rows():
    p = Norm(0, 100)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    assert (p.dweight == 0).all()


@pytest.mark.gpu
def test_in_place():
    """h over r, dx over dh: each lane writes what it read itself."""
    p, q = Norm(50, 3000, seed=3), Norm(50, 3000, seed=3)
    p.forward()
    p.backward()
    plan = migemm.NormPlan(50, 3000, EPS, BF16, x_rs=q.x.stride(0), y_rs=q.x.stride(0),
                           r_rs=q.r.stride(0), h_rs=q.r.stride(0), dy_rs=q.dy.stride(0),
                           dx_rs=q.dh.stride(0), dh_rs=q.dh.stride(0))
    plan.run(q.x, q.r, q.weight, q.r, q.x, None, q.rstd)      # h over r, y over x
    plan.run_backward(q.dy, q.r, q.weight, q.rstd, q.dh, q.dh, q.dweight, q.ws)
    torch.cuda.synchronize()
    assert torch.equal(p.h, q.r) and torch.equal(p.y, q.x) and torch.equal(p.dx, q.dh)
    assert torch.equal(p.dweight, q.dweight)


@pytest.mark.gpu
def test_gradient_against_differences():
    """<dx, v> against central differences of F(h) = sum dy y(h) + sum dh h in
    64 bits along random directions v."""
    p = Norm(11, 350, seed=8)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    ref = p.reference()
    h, w = ref["h"], p.weight.cpu().double()
    dy, dh = p.dy.cpu().double(), p.dh.cpu().double()

    def value(at, weight):
        n = at * (at.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        return (dy * n * weight).sum() + (dh * at).sum()

    g = torch.Generator().manual_seed(1)
    t = 1e-6
    bound = 2.0 ** -8 * ref["dx"].abs() + 2 * SUM * ref["dx_size"]
    for _ in range(4):
        v = torch.randn(h.shape, generator=g, dtype=torch.float64)
        diff = (value(h + t * v, w) - value(h - t * v, w)) / (2 * t)
        got = (p.dx.cpu().double() * v).sum()
        assert abs(got - diff) <= (bound * v.abs()).sum() + 1e-6 * ref["dx_size"].sum()
        u = torch.randn(w.shape, generator=g, dtype=torch.float64)
        diff = (value(h, w + t * u) - value(h, w - t * u)) / (2 * t)
        got = (p.dweight.cpu().double() * u).sum()
        assert abs(got - diff) <= 1e-6 * ref["dweight_size"].sum()


@pytest.mark.gpu
def test_runs_agree_on_streams_and_in_a_graph():
    p = Norm(700, 4100, seed=9)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in (p.y, p.h, p.rstd, p.dx, p.dweight)]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(want, (p.y, p.h, p.rstd, p.dx, p.dweight)))

    def spoil():
        for t in (p.y, p.h, p.rstd, p.dx, p.dweight):
            t.fill_(7)
        p.ws.fill_(0xFF)
        torch.cuda.synchronize()

    spoil()
    s = torch.cuda.Stream()
    p.forward(s)
    p.backward(s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward()
        p.backward()
    for _ in range(3):
        spoil()
        graph.replay()
        assert same()
        p.forward()
        p.backward()
        assert same()


@pytest.mark.gpu
def test_run_refusals():
    p = Norm(4, 100)
    lib, plan = migemm.load(), p.plan.handle
    a = [t.data_ptr() for t in (p.x, p.r, p.weight, p.h, p.y)]
    rstd = p.rstd.data_ptr()
    assert lib.gemm_norm_run(plan, a[0], None, a[2], a[3], a[4], None, rstd, None) == BAD
    assert lib.gemm_norm_run(plan, a[0], a[1], a[2], None, a[4], None, rstd, None) == BAD
    assert lib.gemm_norm_run(plan, *a, rstd, rstd, None) == BAD          # a scale for bf16 rows
    assert lib.gemm_norm_run(plan, None, *a[1:], None, rstd, None) == BAD
    assert lib.gemm_norm_run(plan, a[0] + 2, *a[1:], None, rstd, None) == MIS
    assert lib.gemm_norm_run(plan, a[0], a[1], a[2] + 4, a[3], a[4], None, rstd, None) == MIS
    b = [p.dy.data_ptr(), a[3], a[2], rstd, p.dh.data_ptr(), p.dx.data_ptr(), p.dweight.data_ptr()]
    assert lib.gemm_norm_run_backward(plan, *b, None, None) == BAD       # no workspace
    assert lib.gemm_norm_run_backward(plan, *b, p.ws.data_ptr() + 16, None) == MIS
    assert lib.gemm_norm_run_backward(plan, *b[:4], None, *b[5:], p.ws.data_ptr(), None) == BAD
    q = migemm.NormPlan(4, 100, EPS, x_rs=104, y_rs=104)                 # no backward pass
    assert q.workspace_size == 0
    assert lib.gemm_norm_run_backward(q.handle, *b, p.ws.data_ptr(), None) == BAD
    g = migemm.Plan(migemm.make_desc(16, 16, 16, 1, 1, 16, 1, 16, 1, 16, 1, 16, 1))
    assert lib.gemm_norm_run(g.handle, *a, None, rstd, None) == BAD      # another kind of plan
