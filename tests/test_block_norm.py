"""The block norm against its definition in 64 bits: forward in bf16, e4m3 and
int8, gradients, refusals.

Tolerances.  SUM = 80 * 2^-24 covers a sum of positive terms over a row (fewer
than 64 roundings) and the reciprocal root made of it, as test_norm.py derives.
The gate: exp(-|z|) is off by |z| 2^-24 (its argument's rounding) and two units,
the sum, quotient and product by half a unit each: gate(z) = (|z| + 8) 2^-24 of
it, and twice that of its derivative.  Products of these add 2^-24 a factor;
AREA = 8 * 2^-24 covers the ones between two sums.  A bf16 output adds half a
step, 2^-8 of the value, an e4m3 code 2^-4 of it (or 2^-10 among subnormals), an
int8 code half of one."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED
BF16, E4M3, INT8 = migemm.MIGEMM_BF16, migemm.MIGEMM_FP8_E4M3, migemm.MIGEMM_INT8
U = 2.0 ** -24
SUM, AREA = 80 * U, 8 * U
EPS = 1e-5
MATRICES = ("x", "r", "h", "y", "z", "dy", "dx", "dr", "dz", "dh")


def desc(rows=4, cols=100, eps=EPS, branch=1.0, residual=1.0, post=1, y_type=BF16, device=0, **over):
    rs = {k: 104 for k in MATRICES}
    rs.update({k[:-3]: v for k, v in over.items()})
    return migemm.migemm_block_norm_desc(rows, cols, *[rs[k] for k in MATRICES], eps, branch, residual, post, y_type,
                                         device)


def every(v):
    return {k + "_rs": v for k in MATRICES}


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(rows=0), OK), (dict(post=0), OK), (dict(y_type=E4M3, y_rs=112), OK),
    (dict(y_type=INT8, y_rs=112), OK), (dict(branch=0.0, residual=-2.0), OK),
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(post=2), BAD), (dict(post=-1), BAD),
    (dict(y_type=4), BAD), (dict(y_type=0), BAD),
    (dict(eps=0.0), BAD), (dict(eps=-1e-5), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(branch=float("nan")), BAD), (dict(residual=float("inf")), BAD),
    (dict(x_rs=96), BAD), (dict(r_rs=0), BAD), (dict(h_rs=96), BAD), (dict(z_rs=96), BAD),
    (dict(x_rs=100), MIS), (dict(z_rs=100), MIS), (dict(dz_rs=100), MIS), (dict(y_type=INT8), MIS),
    (dict(dy_rs=0), BAD), (dict(dx_rs=0), BAD), (dict(dr_rs=0), BAD), (dict(dz_rs=0), BAD),
    (dict(z_rs=0), BAD),                                             # a gate's gradient without one
    (dict(z_rs=0, dz_rs=0), OK), (dict(dh_rs=0), OK),
    (dict(dy_rs=0, dx_rs=0, dr_rs=0, dz_rs=0), BAD),                 # dh without a backward pass
    (dict(dy_rs=0, dx_rs=0, dr_rs=0, dz_rs=0, dh_rs=0), OK),
    (dict(cols=16384, **every(16384)), OK), (dict(cols=16385, **every(16392)), UNS),
    (dict(x_rs=1 << 61), UNS), (dict(rows=1 << 62), UNS),
])
def test_description_status(over, status):
    assert migemm.gemm_block_norm_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_block_norm_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_block_norm_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_block_norm_run(p, *[None] * 11) == BAD
        assert lib.gemm_block_norm_run_backward(p, *[None] * 16) == BAD
        assert lib.gemm_block_norm_workspace_size(p) == 0
        assert lib.gemm_block_norm_plan_get_info(p, ctypes.byref(info)) == BAD
    assert lib.gemm_block_norm_plan_destroy(None) == OK
    assert lib.gemm_block_norm_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_block_norm_plan_create(None, None) == BAD
    assert lib.gemm_block_norm_desc_validate(None) == BAD


# ---------------------------------------------------------------- GPU plumbing

def strided(rows, cols, dtype, pad):
    """A rows x cols view whose rows start on 16 bytes; the rest is poisoned."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = -(-cols // per) * per + pad * per
    if dtype == torch.int8:
        full = torch.full((rows, ld), 85, dtype=dtype, device="cuda")
    else:
        full = torch.full((rows, ld), float("nan"), device="cuda").to(dtype)
    return full, full[:, :cols]


TYPES = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, INT8: torch.int8}


class Block:
    def __init__(self, rows, cols, y_type=BF16, post=True, gate=True, dh=True, pad=1, seed=0, spread=1.0,
                 branch=0.75, residual=1.25):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.cols, self.y_type, self.post, self.gate = rows, cols, y_type, post, gate
        self.branch, self.residual = branch, residual

        def filled(scale):
            full, v = strided(rows, cols, torch.bfloat16, pad)
            v.copy_((torch.randn(rows, cols, generator=g) * scale).bfloat16())
            return v

        self.x, self.r, self.z = filled(spread), filled(2 * spread), filled(2.0)
        self.dy, self.dh = filled(0.5), filled(0.25)
        self.weight = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16().cuda()
        self.post_weight = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16().cuda() if post else None
        if not gate:
            self.z = None
        if not dh:
            self.dh = None
        self.fulls = {}
        for name in ("y", "h", "dx", "dr") + (("dz",) if gate else ()):
            self.fulls[name], v = strided(rows, cols, TYPES[y_type] if name == "y" else torch.bfloat16, pad)
            setattr(self, name, v)
        if not gate:
            self.dz = None

        def vector(n, used=True):
            return torch.full((n,), float("nan"), device="cuda") if used else None

        self.rstd, self.post_rstd = vector(rows), vector(rows, post)
        self.scale = vector(rows, y_type != BF16)
        self.dweight, self.dpost_weight = vector(cols), vector(cols, post)
        self.make_plan()

    def make_plan(self):
        rs = {k + "_rs": m.stride(0) for k in MATRICES if (m := getattr(self, k)) is not None}
        self.plan = migemm.BlockNormPlan(self.rows, self.cols, EPS, self.y_type, post_norm=self.post,
                                         branch_scale=self.branch, residual_scale=self.residual, **rs)
        self.ws = torch.full((self.plan.workspace_size,), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        self.plan.run(self.x, self.z, self.r, self.post_weight, self.weight, self.h, self.y, self.scale,
                      self.post_rstd, self.rstd, stream)

    def backward(self, stream=None):
        self.plan.run_backward(self.dy, self.dh, self.x, self.z, self.h, self.post_weight, self.weight,
                               self.post_rstd, self.rstd, self.dx, self.dz, self.dr, self.dpost_weight, self.dweight,
                               self.ws, stream)

    def outputs(self):
        return [t for t in (self.h, self.y, self.scale, self.rstd, self.post_rstd, self.dx, self.dz, self.dr,
                            self.dweight, self.dpost_weight) if t is not None]


def d(t):
    return t.cpu().double()


def within(got, want, bound, what=""):
    got = d(got)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (what, over.max().item(), over.argmax().item())


def gate_of(z):
    """sigmoid(z), its derivative and how far off the kernels may have them, relative."""
    e = torch.exp(-z.abs())
    s = torch.where(z < 0, e / (1 + e), 1 / (1 + e))
    return s, e / (1 + e) ** 2, (z.abs() + 8) * U


def check(p):
    x, w = d(p.x), d(p.weight)
    if p.post:
        post = (x.pow(2).mean(1) + EPS).rsqrt()
        within(p.post_rstd, post, SUM * post, "post_rstd")
        u = x * post[:, None] * d(p.post_weight)
    else:
        u = x
    off = (SUM if p.post else 0) + AREA
    if p.gate:
        s, _, rel = gate_of(d(p.z))
        u, off = u * s, off + rel
    a, b = p.branch * u, p.residual * d(p.r)
    h, h_off = a + b, a.abs() * off + (a.abs() + b.abs()) * 2 * U
    within(p.h, h, 2.0 ** -8 * (h.abs() + h_off) + h_off + 1e-38, "h")
    square = h.pow(2).mean(1) + EPS
    rstd = square.rsqrt()
    rel = SUM + (h.abs() * h_off).mean(1) / square
    within(p.rstd, rstd, rel * rstd, "rstd")
    y = h * rstd[:, None] * w
    y_off = y.abs() * (rel + AREA)[:, None] + h_off * rstd[:, None] * w.abs()
    if p.y_type == BF16:
        within(p.y, y, 2.0 ** -8 * (y.abs() + y_off) + y_off + 1e-38, "y")
        return
    top = 448 if p.y_type == E4M3 else 127
    largest, s_off = y.abs().amax(1), y_off.amax(1)
    within(p.scale, largest / top, (s_off + largest * AREA) / top + 1e-44, "scale")
    some = largest > 0
    over = torch.where(some, largest, 1.0)[:, None]
    q = torch.where(some[:, None], y / over * top, 0.0)
    q_off = torch.where(some[:, None], (y_off + y.abs() * (s_off / over[:, 0] + AREA)[:, None]) / over * top, 0.0)
    if p.y_type == E4M3:
        q_off += torch.maximum(2.0 ** -4 * (q.abs() + q_off), torch.tensor(2.0 ** -10, dtype=torch.float64))
    else:
        q_off += 0.5
    within(p.y.float(), q, q_off, "codes")
    assert (p.y.float().abs().amax(1).cpu()[some] == top).all()


def gradients(p):
    """From what the forward pass stored: the gradients, and the sizes and errors of their terms."""
    h, w, g = d(p.h), d(p.weight), d(p.dy)
    rstd = d(p.rstd)[:, None]
    n = h * rstd
    gwn = g * w * n
    dh = d(p.dh) if p.dh is not None else torch.zeros_like(h)
    dd = dh + rstd * (g * w - n * gwn.mean(1, keepdim=True))
    d_off = 2 * SUM * (dh.abs() + rstd * ((g * w).abs() + n.abs() * gwn.abs().mean(1, keepdim=True)))
    out = {"dr": (p.residual * dd, abs(p.residual) * d_off), "dweight": ((g * n).sum(0), 0 * w, (g * n).abs().sum(0))}
    v, v_off = p.branch * dd, abs(p.branch) * d_off
    x = d(p.x)
    post = d(p.post_rstd)[:, None] if p.post else 1.0
    pw = d(p.post_weight) if p.post else 1.0
    px = x * post
    if p.gate:
        s, ds, rel = gate_of(d(p.z))
        u = px * pw
        dz = v * u * ds
        out["dz"] = (dz, v_off * (u * ds).abs() + dz.abs() * (2 * rel + AREA))
        v, v_off = v * s, v_off * s + v.abs() * s * (rel + U)
    if p.post:
        out["dpost_weight"] = ((v * px).sum(0), (v_off * px.abs()).sum(0), ((v.abs() + v_off) * px.abs()).sum(0))
        t, t_off = v * pw, v_off * pw.abs()
        m = (t * px).mean(1, keepdim=True)
        m_off = (t_off * px.abs()).mean(1, keepdim=True) + SUM * (t * px).abs().mean(1, keepdim=True)
        v_off = post * (t_off + px.abs() * m_off) + AREA * post * (t.abs() + (px * m).abs())
        v = post * (t - px * m)
    out["dx"] = (v, v_off)
    return out


def check_backward(p):
    for name, (want, off, *size) in gradients(p).items():
        if size:  # fp32 sums: rows / walkers additions a walker, then 48 over the partial rows
            within(getattr(p, name), want, off + (p.rows / 512 + 100) * U * size[0] + 1e-38, name)
        else:
            within(getattr(p, name), want, 2.0 ** -8 * (want.abs() + off) + off + 1e-38, name)


def untouched(p):
    for n, full in p.fulls.items():
        rest = full[:, p.cols:]
        assert ((rest == 85) if rest.dtype == torch.int8 else torch.isnan(rest.float())).all(), n


SHAPES = [(1, 1), (1, 8192), (3, 7), (5, 64), (300, 511), (37, 512), (9, 513), (70, 1024), (6, 1031),
          (129, 2048), (4, 2049), (33, 5000), (1030, 300), (2, 8193), (3, 16384), (600, 4096), (300, 8192),
          (300, 12000), (1100, 1500), (2000, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("post", [True, False], ids=["post", "bare"])
@pytest.mark.parametrize("gate", [True, False], ids=["gate", "open"])
def test_forward_and_gradients(rows, cols, post, gate):
    p = Block(rows, cols, BF16, post, gate, dh=(rows + cols) % 3 != 0, seed=rows * 7 + cols)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p)
    check_backward(p)
    untouched(p)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("y_type,post,gate", [(E4M3, True, True), (INT8, True, False), (INT8, False, True),
                                              (E4M3, False, False)])
def test_codes(rows, cols, y_type, post, gate):
    p = Block(rows, cols, y_type, post, gate, seed=rows * 3 + cols)
    p.forward()
    torch.cuda.synchronize()
    check(p)
    assert (p.fulls["y"][:, cols:].view(torch.uint8) == p.fulls["y"][0, -1].view(torch.uint8)).all()
    assert torch.isnan(p.fulls["h"][:, cols:].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-18, 1e-3, 1e4, 1e15])
@pytest.mark.parametrize("y_type", [BF16, E4M3, INT8], ids=["bf16", "e4m3", "int8"])
def test_magnitudes(spread, y_type):
    """With a gate alone, so that the second norm sees them."""
    p = Block(20, 777, y_type, post=False, seed=5, spread=spread)
    p.forward()
    torch.cuda.synchronize()
    check(p)


@pytest.mark.gpu
@pytest.mark.parametrize("branch,residual", [(0.0, 1.0), (1.0, 0.0), (-0.5, 2.0)])
def test_scales(branch, residual):
    p = Block(40, 600, seed=6, branch=branch, residual=residual)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p)
    check_backward(p)


@pytest.mark.gpu
def test_gates_at_their_ends():
    """sigmoid(z) for z from -infinity to infinity: no NaN, and 0 and 1 there."""
    p = Block(4, 64, seed=2)
    p.z[0] = float("-inf")
    p.z[1] = float("inf")
    p.z[2] = -200.0
    p.z[3] = torch.linspace(-95, 95, 64).bfloat16().cuda()
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    for t in (p.h, p.y, p.dx, p.dz, p.dr):
        assert torch.isfinite(t.float()).all()
    r = (p.residual * p.r[0].float()).bfloat16()
    assert torch.equal(p.h[0], r) and (p.dx[0] == 0).all() and (p.dz[:2] == 0).all()
    p.z[:2] = 0                                            # (the definition's sizes hold no infinity)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p)
    check_backward(p)


@pytest.mark.gpu
def test_rows_of_zeros_nan_and_infinity():
    for y_type in (BF16, E4M3, INT8):
        p = Block(6, 600, y_type, gate=False, seed=1)
        p.x[1] = 0
        p.r[1] = 0
        p.x[2, 599] = float("nan")
        p.r[3, 0] = float("inf")
        p.x[4] = 1e-40                                     # bf16 subnormals
        p.forward()
        torch.cuda.synchronize()
        y = p.y.float().cpu()
        assert (y[1] == 0).all() and torch.isfinite(y[[0, 1, 4, 5]]).all()
        if y_type == BF16:
            assert torch.isnan(y[2]).all() and torch.isnan(y[3, 0])
            continue
        scale = p.scale.cpu()
        assert scale[1] == 0 and not torch.isfinite(scale[2:4]).any() and torch.isfinite(scale[[0, 4, 5]]).all()
        if y_type == INT8:
            assert torch.isnan(scale[2:4]).all() and (y[2:4] == 0).all()


@pytest.mark.gpu
def test_no_rows():
    p = Block(0, 100)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    assert (p.dweight == 0).all() and (p.dpost_weight == 0).all()


@pytest.mark.gpu
def test_in_place():
    """h over r, y over x; dr over dh, dx over dy, dz over z: each lane writes
    what it read itself."""
    p, q = Block(50, 3000, seed=3), Block(50, 3000, seed=3)
    p.forward()
    p.backward()
    x, z = q.x.clone(), q.z.clone()
    q.h, q.y = q.r, q.x
    q.make_plan()
    q.forward()
    torch.cuda.synchronize()
    assert torch.equal(p.h, q.h) and torch.equal(p.y, q.y)
    q.x, q.z = torch.empty_like(p.fulls["y"])[:, :3000].copy_(x), torch.empty_like(p.fulls["y"])[:, :3000].copy_(z)
    q.dr, q.dx, q.dz = q.dh, q.dy, q.z
    q.make_plan()
    q.backward()
    torch.cuda.synchronize()
    for n in ("dx", "dz", "dr", "dweight", "dpost_weight"):
        assert torch.equal(getattr(p, n), getattr(q, n)), n


@pytest.mark.gpu
def test_without_x_where_nothing_needs_it():
    p = Block(30, 500, post=False, gate=False, seed=4)
    p.forward()
    p.plan.run_backward(p.dy, p.dh, None, None, p.h, None, p.weight, None, p.rstd, p.dx, None, p.dr, None, p.dweight,
                        p.ws)
    torch.cuda.synchronize()
    check_backward(p)


@pytest.mark.gpu
@pytest.mark.parametrize("post", [True, False], ids=["post", "bare"])
def test_gradient_against_differences(post):
    """<gradient, v> against central differences of F = sum dy y + sum dh h in
    64 bits along random directions of x, z, r and the weights.  The kernels
    take h as it was stored, half a step from F's: n is off by 2^-8 of it, and
    what n stands in twice by twice that."""
    p = Block(11, 350, post=post, seed=8)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    dy, dh = d(p.dy), d(p.dh)
    at = {"x": d(p.x), "z": d(p.z), "r": d(p.r), "w": d(p.weight)}
    if post:
        at["pw"] = d(p.post_weight)

    def value(a):
        u = a["x"]
        if post:
            u = u * (u.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * a["pw"]
        h = p.residual * a["r"] + p.branch * torch.sigmoid(a["z"]) * u
        return (dy * h * (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * a["w"]).sum() + (dh * h).sum()

    # What the stored h's rounding does to d, and d's error to each gradient.
    h, w, rstd = d(p.h), d(p.weight), d(p.rstd)[:, None]
    n = h * rstd
    stored = 2.0 ** -8 * rstd * 2 * n.abs() * ((dy * w * n).abs().mean(1, keepdim=True))
    s, ds, _ = gate_of(at["z"])
    k = d(p.post_rstd)[:, None] if post else 1.0
    pw = at["pw"] if post else 1.0
    px = at["x"] * k
    through = abs(p.branch) * stored * s
    t = (through * pw if not post else through * pw.abs())
    by = {"r": abs(p.residual) * stored, "z": abs(p.branch) * stored * (px * pw * ds).abs(), "w": None,
          "x": t if not post else k * (t + px.abs() * (t * px.abs()).mean(1, keepdim=True))}
    by["w"] = (2.0 ** -8 * (dy * n).abs()).sum(0)
    by["pw"] = (through * px.abs()).sum(0)
    names = {"x": "dx", "z": "dz", "r": "dr", "w": "dweight", "pw": "dpost_weight"}
    got = gradients(p)
    g, step = torch.Generator().manual_seed(1), 1e-6
    for name in at:
        want, off, *size = got[names[name]]
        bound = by[name] + off + ((p.rows / 512 + 100) * U * size[0] if size else 2.0 ** -8 * (want.abs() + off))
        for _ in range(3):
            v = torch.randn(at[name].shape, generator=g, dtype=torch.float64)
            hi, lo = ({**at, name: at[name] + sign * step * v} for sign in (1, -1))
            diff = (value(hi) - value(lo)) / (2 * step)
            mine = (d(getattr(p, names[name])) * v).sum()
            assert abs(mine - diff) <= (bound * v.abs()).sum() + 1e-6 * want.abs().sum(), name


@pytest.mark.gpu
@pytest.mark.parametrize("y_type", [BF16, INT8], ids=["bf16", "int8"])
def test_runs_agree_on_streams_and_in_a_graph(y_type):
    p = Block(700, 4100, y_type, seed=9)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in p.outputs()]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))
                   for a, b in zip([w.contiguous() for w in want], p.outputs()))

    def spoil():
        for t in p.outputs():
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
@pytest.mark.parametrize("rows,cols,forward,backward", [
    (5, 512, (1, 1), (1, 1)), (2000, 500, (1, 1), (1, 1)), (300, 1001, (1, 2), (1, 2)), (300, 2000, (1, 4), (4, 1)),
    (5, 2048, (4, 1), (4, 1)), (300, 4001, (4, 2), (4, 2)), (300, 8190, (4, 4), (8, 2)), (3, 8001, (16, 1), (16, 1)),
    (40, 16383, (8, 4), (8, 4)), (700, 12001, (8, 4), (8, 4)),
    # (even and odd numbers of columns have kernels of their own)
    (5, 511, (1, 1), (1, 1)), (300, 1000, (1, 2), (1, 2)), (300, 1999, (1, 4), (4, 1)), (5, 2047, (4, 1), (4, 1)),
    (300, 4000, (4, 2), (4, 2)), (300, 8191, (4, 4), (8, 2)), (3, 8000, (16, 1), (16, 1)), (40, 16382, (8, 4), (8, 4))])
def test_kernels_that_a_plan_chooses(rows, cols, forward, backward):
    for gate, post in ((True, True), (False, True), (True, False), (False, False)):
        p = Block(rows, cols, post=post, gate=gate, seed=rows + cols)
        i = p.plan.info
        assert (i.forward_waves, i.forward_vectors) == forward and (i.backward_waves, i.backward_vectors) == backward
        assert i.backward_workgroups * cols * (1 + post) * 4 == p.plan.workspace_size
        p.forward()
        p.backward()
        torch.cuda.synchronize()
        check(p)
        check_backward(p)
        untouched(p)


@pytest.mark.gpu
def test_run_refusals():
    p = Block(4, 100, E4M3)
    lib, plan = migemm.load(), p.plan.handle
    f = [t.data_ptr() for t in (p.x, p.z, p.r, p.post_weight, p.weight, p.h, p.y, p.scale, p.post_rstd, p.rstd)]
    for i in range(10):
        a = list(f)
        a[i] = None
        assert lib.gemm_block_norm_run(plan, *a, None) == BAD, i
        a[i] = f[i] + 2
        assert lib.gemm_block_norm_run(plan, *a, None) == MIS, i
    b = [t.data_ptr() for t in (p.dy, p.dh, p.x, p.z, p.h, p.post_weight, p.weight, p.post_rstd, p.rstd, p.dx, p.dz,
                                p.dr, p.dpost_weight, p.dweight, p.ws)]
    for i in range(15):
        a = list(b)
        a[i] = None
        assert lib.gemm_block_norm_run_backward(plan, *a, None) == BAD, i
        a[i] = b[i] + 2
        assert lib.gemm_block_norm_run_backward(plan, *a, None) == MIS, i
    q = Block(4, 100, post=False, gate=False, dh=False)                     # what such a plan has not is refused
    f = [q.x.data_ptr(), None, q.r.data_ptr(), None, q.weight.data_ptr(), q.h.data_ptr(), q.y.data_ptr(), None, None,
         q.rstd.data_ptr()]
    for i in (1, 3, 7, 8):
        a = list(f)
        a[i] = q.x.data_ptr()
        assert lib.gemm_block_norm_run(q.plan.handle, *a, None) == BAD, i
    n = migemm.BlockNormPlan(4, 100, EPS, x_rs=104, r_rs=104, h_rs=104, y_rs=104)   # no backward pass
    assert n.workspace_size == 0
    assert lib.gemm_block_norm_run_backward(n.handle, *b, None) == BAD
    m = migemm.NormPlan(4, 100, EPS, x_rs=104, y_rs=104)
    assert lib.gemm_block_norm_run(m.handle, *f, None) == BAD               # another kind of plan
