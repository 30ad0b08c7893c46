"""The operators on matrices past 4 GiB, each role in turn: what the rows on
both sides of 2^31 and 2^32 bytes, the first and the last ones give, against 64
bits (tolerances: test_norm.py's, test_scaled_kernels.py's and
test_vocab_loss.py's).  Where a sum runs over all rows, all but those rows add
zeros to it, so that its tolerance is that of a short sum."""
import pytest
import torch

from tests.test_norm import EPS, SUM
from tests.test_scaled_kernels import largest_of_octets
from tests.test_vocab_loss import U, within
from warp_specialized_pipelined_amd import migemm

pytestmark = pytest.mark.gpu


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("needs %d GiB" % gib)


def around(rows, row_bytes):
    """Row numbers to look at: the ends, and those beside 2^31 and 2^32 bytes."""
    at = {0, 1, rows // 2, rows - 2, rows - 1}
    for edge in (1 << 31, 1 << 32):
        at.update(r for r in range(edge // row_bytes - 2, edge // row_bytes + 3) if 0 <= r < rows)
    return torch.tensor(sorted(at), device="cuda")


def normal(rows, cols, scale=1.0, dtype=torch.bfloat16):
    """Filled a part at a time."""
    t = torch.empty(rows, cols, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        t[r:r + n] = (torch.randn(n, cols, generator=g, device="cuda") * scale).to(dtype)
    return t


def only(t, at):
    """t with zeros in every row but those."""
    keep = t[at].clone()
    t.zero_()
    t[at] = keep
    return t


def test_norm():
    need(60)
    rows, cols = 70000, 32768
    at = around(rows, 2 * cols)
    x, r, dh = normal(rows, cols), normal(rows, cols, 2.0), normal(rows, cols, 0.25)
    dy = only(normal(rows, cols, 0.5), at)
    weight = (1 + 0.3 * torch.randn(cols, device="cuda")).bfloat16()
    h, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, dweight = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    plan = migemm.NormPlan(rows, cols, EPS, x_rs=cols, y_rs=cols, r_rs=cols, h_rs=cols, dy_rs=cols, dx_rs=cols,
                           dh_rs=cols)
    ws = torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    plan.run(x, r, weight, h, y, None, rstd)
    plan.run_backward(dy, h, weight, rstd, dh, dx, dweight, ws)
    torch.cuda.synchronize()
    hs = (x[at].double() + r[at].double()).bfloat16()
    assert torch.equal(h[at], hs)
    hs, w, g = hs.double(), weight.double(), dy[at].double()
    want = (hs.pow(2).mean(1) + EPS).rsqrt()
    n = hs * want[:, None]
    within(rstd[at], want, SUM * want)
    within(y[at], n * w, (2.0 ** -8 + SUM) * (n * w).abs() + 1e-38)
    d = want[:, None] * (g * w - n * (g * w * n).mean(1, keepdim=True)) + dh[at].double()
    size = want[:, None] * ((g * w).abs() + n.abs() * (g * w * n).abs().mean(1, keepdim=True)) + dh[at].double().abs()
    within(dx[at], d, 2.0 ** -8 * d.abs() + 2 * SUM * size + 1e-38)
    # at most one row that is not zero for most walkers, then 48 additions (and a row or two more)
    within(dweight, (g * n).sum(0), 128 * 2.0 ** -24 * (g * n).abs().sum(0) + 1e-38)


@pytest.mark.parametrize("M,N,K", [(600000, 40, 8000), (3, 600000, 8000), (150, 600000, 8000)])
def test_scaled(M, N, K):
    need(40)
    a, b = (normal(n, K, 60.0, torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    ld = -(-N // 8) * 8
    d = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")
    plan = migemm.ScaledPlan(M, N, K, a_rs=K, b_cs=K, d_rs=ld)
    ws = torch.empty(plan.workspace_size + 256, dtype=torch.uint8, device="cuda")
    plan.run(a, sa, b, sb, d, ws)
    torch.cuda.synchronize()
    rows = around(M, K) if M > 1000 else torch.arange(M, device="cuda")
    cols = around(N, K) if N > 1000 else torch.arange(N, device="cuda")
    x, z = a.view(torch.uint8)[rows].view(a.dtype), b.view(torch.uint8)[cols].view(b.dtype)
    scale = sa[rows].double()[:, None] * sb[cols].double()
    u, v = x.float().double(), z.float().double()
    want, size = (u @ v.t()) * scale, (u.abs() @ v.abs().t()) * scale
    err = (K + 4) * 2.0 ** -23 * size + 7 * 2.0 ** -13 * largest_of_octets(x, z) * scale
    within(d[rows][:, cols], want, err + 2.0 ** -8 * (want.abs() + err))


@pytest.mark.parametrize("T,V,H", [(600000, 200, 4000), (5, 600000, 4000), (2200000, 1024, 64)])
def test_vocab_loss(T, V, H):
    """x and dx, w and dw, and g (of 2200000 rows, 4.8 GB) past 4 GiB."""
    need(60)
    row_bytes = 2 * (1088 if T > 1 << 20 else H)
    rows = around(T, row_bytes) if T > 1000 else torch.arange(T, device="cuda")
    cols = around(V, 2 * H) if V > 2000 else torch.arange(V, device="cuda")
    x, w = normal(T, H), normal(V, H, 2.0 / H ** 0.5)
    if T > 1000:
        only(x, rows)
    g = torch.Generator(device="cuda").manual_seed(5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[:: 7] = -100
    target[rows[0]], target[rows[-1]] = 0, V - 1
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    plan = migemm.VocabLossPlan(T, V, H, x_rs=H, w_rs=H, dx_rs=H, dw_rs=H)
    ws = torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    plan.run(x, w, target, loss, lse, ws)
    plan.run_backward(x, w, target, lse, dloss, dx, dw, ws)
    torch.cuda.synchronize()
    counts, at = target[rows] >= 0, target[rows].clamp(min=0)
    xs = x[rows].double()
    logits = torch.cat([xs @ w[c:c + 65536].double().t() for c in range(0, V, 65536)], 1)
    L = (H + 4) * U * torch.cat([(xs.abs() @ w[c:c + 65536].double().abs().t()).amax(1, keepdim=True)
                                 for c in range(0, V, 65536)], 1).amax(1)
    want = torch.logsumexp(logits, 1)
    within(lse[rows], want, L + 256 * U + 4 * U * want.abs())
    picked = logits.gather(1, at[:, None]).squeeze(1)
    within(loss[rows], torch.where(counts, want - picked, 0.0),
           torch.where(counts, 2 * L + 256 * U + 6 * U * (want.abs() + picked.abs()), 0.0))
    p = torch.softmax(logits, 1)
    dl = torch.where(counts, dloss[rows].double(), 0.0)[:, None]
    gs = p.clone()
    gs[torch.arange(len(rows), device="cuda"), at] -= 1
    gs *= dl
    R = (2 * L + 512 * U + 8 * U * want.abs())[:, None]
    gerr = R * p * dl + 2.0 ** -8 * (gs.abs() + R * p * dl)

    def check(got, terms, n):
        ref, mag, err = (sum(t[i] for t in terms) for i in range(3))
        within(got, ref, err + (n + 8) * U * (mag + err) + 2.0 ** -8 * (ref.abs() + err) + 1e-38)

    check(dx[rows], [(gs[:, c:c + 65536].contiguous() @ w[c:c + 65536].double(),
                      gs[:, c:c + 65536].abs().contiguous() @ w[c:c + 65536].double().abs(),
                      gerr[:, c:c + 65536].contiguous() @ w[c:c + 65536].double().abs()) for c in range(0, V, 65536)], V)
    gc, ec = gs[:, cols].t().contiguous(), gerr[:, cols].t().contiguous()
    check(dw[cols], [(gc @ xs, gc.abs() @ xs.abs(), ec @ xs.abs())], len(rows))
    assert (dx[target < 0] == 0).all()
