"""The int8 product, the rows to 8 bits, the block norm and the checkpoint on
matrices past 4 GiB, each role in turn: what the rows on both sides of 2^31 and
2^32 bytes, the first and the last ones give, against 64 bits (tolerances: those
of test_int8.py, test_quantize.py, test_block_norm.py and test_checkpoint.py).
Where a sum runs over all rows, all but those rows add zeros to it, so that its
tolerance is that of a short sum."""
import pytest
import torch

from tests.test_block_norm import AREA, EPS, SUM, U, gate_of, within
from tests.test_checkpoint import packed, power
from tests.test_operators_past_32_bits import around, need, normal, only
from warp_specialized_pipelined_amd import migemm

pytestmark = pytest.mark.gpu


def codes(rows, cols):
    t = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        t[r:r + n] = torch.randint(-128, 128, (n, cols), generator=g, device="cuda", dtype=torch.int8)
    return t


@pytest.mark.parametrize("M,N,K", [(600000, 40, 8000), (3, 600000, 8000), (150, 600000, 8000)])
def test_int8(M, N, K):
    need(40)
    a, b = codes(M, K), codes(N, K)
    sa, sb = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    bias = torch.randn(N, device="cuda") * 1e5
    ld = -(-N // 8) * 8
    d = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")
    plan = migemm.Int8Plan(M, N, K, a_rs=K, b_cs=K, d_rs=ld)
    ws = torch.empty(plan.workspace_size + 256, dtype=torch.uint8, device="cuda")
    plan.run(a, sa, b, sb, bias, d, ws)
    torch.cuda.synchronize()
    rows = around(M, K) if M > 1000 else torch.arange(M, device="cuda")
    cols = around(N, K) if N > 1000 else torch.arange(N, device="cuda")
    term = (a[rows].double() @ b[cols].double().t()) * sa[rows].double()[:, None] * sb[cols].double()
    want = term + bias[cols].double()
    off = 5 * U * (term.abs() + bias[cols].double().abs())
    within(d[rows][:, cols], want.cpu(), (off + 2.0 ** -8 * (want.abs() + off)).cpu())


def test_quantize():
    need(30)
    rows, cols = 300000, 16384
    at = around(rows, cols)
    at = torch.unique(torch.cat([at, around(rows, 2 * cols)]))
    x = normal(rows, cols)
    q, scale = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    migemm.QuantizePlan(rows, cols, x_rs=cols, q_rs=cols).run(x, q, scale)
    torch.cuda.synchronize()
    xs = x[at].double()
    largest = xs.abs().amax(1)
    assert torch.equal(q[at].double(), torch.round(xs * 127 / largest[:, None]))
    assert ((scale[at].double() - largest / 127).abs() <= U * largest / 127).all()


def test_block_norm():
    need(90)
    rows, cols = 150000, 16384
    at = around(rows, 2 * cols)
    x, r, z, dh = normal(rows, cols), normal(rows, cols, 2.0), normal(rows, cols, 1.5), normal(rows, cols, 0.25)
    dy = only(normal(rows, cols, 0.5), at)
    only(dh, at)
    w, pw = ((1 + 0.3 * torch.randn(cols, device="cuda")).bfloat16() for _ in range(2))
    h, y, dx, dz, dr = (torch.empty_like(x) for _ in range(5))
    rstd, post = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, dpw = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    rs = {k + "_rs": cols for k in ("x", "r", "h", "y", "z", "dy", "dx", "dr", "dz", "dh")}
    plan = migemm.BlockNormPlan(rows, cols, EPS, **rs)
    ws = torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    plan.run(x, z, r, pw, w, h, y, None, post, rstd)
    plan.run_backward(dy, dh, x, z, h, pw, w, post, rstd, dx, dz, dr, dpw, dw, ws)
    torch.cuda.synchronize()

    def of(t):
        return t[at].cpu().double()

    xs, s_off = of(x), gate_of(of(z))
    s, ds, rel = s_off
    want = (xs.pow(2).mean(1) + EPS).rsqrt()
    within(post[at], want, SUM * want, "post_rstd")
    wd, pwd = w.cpu().double(), pw.cpu().double()
    u = xs * want[:, None] * pwd * s
    hs, off = of(r) + u, u.abs() * (SUM + AREA + rel) + (u.abs() + of(r).abs()) * 2 * U
    within(h[at], hs, 2.0 ** -8 * (hs.abs() + off) + off, "h")
    root = (hs.pow(2).mean(1) + EPS).rsqrt()
    within(rstd[at], root, 2 * SUM * root, "rstd")
    n = of(h) * of(rstd)[:, None]
    g = of(dy)
    gwn = g * wd * n
    k = of(rstd)[:, None]
    d = of(dh) + k * (g * wd - n * gwn.mean(1, keepdim=True))
    d_off = 2 * SUM * (of(dh).abs() + k * ((g * wd).abs() + n.abs() * gwn.abs().mean(1, keepdim=True)))
    within(dr[at], d, 2.0 ** -8 * (d.abs() + d_off) + d_off, "dr")
    px = xs * of(post)[:, None]
    v = d * px * pwd * ds
    v_off = d_off * (px * pwd * ds).abs() + v.abs() * (2 * rel + AREA)
    within(dz[at], v, 2.0 ** -8 * (v.abs() + v_off) + v_off, "dz")
    # at most one row that is not zero for most walkers, then 48 additions (and a row or two more)
    within(dw, (g * n).sum(0), 128 * U * (g * n).abs().sum(0) + 1e-38, "dweight")
    t = d * s * px
    t_off = (d_off * s + t.abs() * (rel + AREA)) * px.abs().clamp(min=1)
    within(dpw, t.sum(0), 128 * U * t.abs().sum(0) + 2 * t_off.sum(0) + 1e-38, "dpost_weight")


@pytest.mark.parametrize("T,C,N,dw_type", [(600000, 8000, 40, migemm.MIGEMM_BF16), (600000, 40, 4000, migemm.MIGEMM_FP32),
                                           (50, 4000, 600000, migemm.MIGEMM_FP32),
                                           (50, 600000, 8000, migemm.MIGEMM_BF16)])
def test_checkpoint(T, C, N, dw_type):
    """x and the kept form, dy, and dw (of many rows, and of long ones) past 4 GiB."""
    need(60)
    at = around(T, 2 * C) if T * C > T * N else around(T, 2 * N)
    if T * C > T * N:
        at = torch.unique(torch.cat([at, around(T, C)]))  # the codes' own rows of bytes
    x, dy = normal(T, C), normal(T, N, 0.5)
    if T > 1000:
        only(x, at)
    ld = C
    dw = torch.empty(N, ld, dtype=torch.float32 if dw_type == migemm.MIGEMM_FP32 else torch.bfloat16, device="cuda")
    plan = migemm.CheckpointPlan(T, C, x_rs=C, out_cols=N, dy_rs=N, dw_rs=ld, dw_type=dw_type)
    kept = torch.empty(plan.checkpoint_size, dtype=torch.uint8, device="cuda")
    ws = torch.empty(plan.workspace_size + 256, dtype=torch.uint8, device="cuda")
    plan.pack(x, kept)
    back = torch.full_like(x, 7)
    plan.unpack(kept, back)
    plan.weight_gradient(dy, kept, dw, ws)
    torch.cuda.synchronize()
    # What came back is the definition's, in the groups of 32 tokens those rows are in.
    group = torch.unique(at // 32)
    rows = (group[:, None] * 32 + torch.arange(32, device="cuda")).flatten()
    rows = rows[rows < T]
    if T > 1000:
        assert T % 32 == 0
        some = torch.arange(C, device="cuda")
    else:
        some = torch.cat([torch.arange(40, device="cuda"), torch.arange(C - 40, C, device="cuda")])
    values, e = packed(x[rows][:, some])
    exact = (values * power(e - 127)[:, None]).reshape(-1, values.shape[2])[:len(rows), :len(some)]
    assert torch.equal(back[rows][:, some].double().cpu(), exact)
    cols = torch.arange(C, device="cuda") if C <= 8000 else around(C, 2)
    outs = torch.arange(N, device="cuda") if N <= 4000 else around(N, (4 if dw_type == migemm.MIGEMM_FP32 else 2) * ld)
    xs, ds = back[rows][:, cols].double(), dy[rows][:, outs].double()
    want, size = ds.t().contiguous() @ xs, ds.abs().t().contiguous() @ xs.abs()
    off = (len(rows) + 4) * 2.0 ** -23 * size
    if dw_type == migemm.MIGEMM_BF16:
        off = off + 2.0 ** -8 * (want.abs() + off)
    over = (dw[outs][:, cols].double() - want).abs() - off - 1e-38
    assert (over <= 0).all(), over.max().item()
