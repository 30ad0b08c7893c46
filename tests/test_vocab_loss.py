"""The vocabulary loss against its definition in 64 bits.

Tolerances.  With u = 2^-24 and D a row's largest sum of |x w| over a logit:
  logits: off by at most L = (H + 4) u D;
  lse: moves by at most L, plus the roundings of a sum of positive terms (64
    a lane, then joins over lanes, parts of the vocabulary and 64 threads:
    fewer than 256) and of its logarithm: L + 256 u + 4 u |lse|;
  loss: another L, and a rounding of the difference;
  p = exp(logit - lse): relative error R = 2 L + 512 u + 8 u |lse|;
  g: p's error times dloss, and its rounding to bf16, 2^-8 |g|;
  dx, dw: that summed against |w| or |x|, an fp32 sum of n terms (n u of the
    sum of magnitudes), and half a bf16 step, 2^-8, of the result."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

OK, BAD = migemm.MIGEMM_OK, migemm.MIGEMM_ERR_INVALID_ARG
MIS, UNS = migemm.MIGEMM_ERR_MISALIGNED, migemm.MIGEMM_ERR_UNSUPPORTED
U = 2.0 ** -24


def desc(rows=5, vocab=100, hidden=60, x_rs=64, w_rs=64, dx_rs=64, dw_rs=64, device=0, reserved=0):
    return migemm.migemm_vocab_loss_desc(rows, vocab, hidden, x_rs, w_rs, dx_rs, dw_rs, device, reserved)


@pytest.mark.parametrize("over,status", [
    (dict(), OK),
    (dict(rows=0), OK),
    (dict(rows=-1), BAD), (dict(vocab=0), BAD), (dict(hidden=0), BAD), (dict(vocab=-4), BAD),
    (dict(reserved=1), BAD),
    (dict(x_rs=56), BAD), (dict(w_rs=0), BAD), (dict(dx_rs=56), BAD), (dict(dw_rs=8), BAD),
    (dict(x_rs=60), MIS), (dict(w_rs=62), MIS), (dict(dx_rs=68), MIS), (dict(dw_rs=63), MIS),
    (dict(dx_rs=0), BAD), (dict(dw_rs=0), BAD), (dict(dx_rs=0, dw_rs=0), OK),
    (dict(rows=1 << 28), UNS), (dict(vocab=1 << 28), UNS),
    (dict(x_rs=1 << 22), UNS), (dict(w_rs=1 << 22), UNS), (dict(dx_rs=1 << 22), UNS),
    (dict(dw_rs=1 << 60), UNS), (dict(rows=1 << 61), UNS),
])
def test_description_status(over, status):
    assert migemm.gemm_vocab_loss_desc_validate(desc(**over)) == status


def test_calls_refuse_what_is_not_a_loss_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_vocab_loss_run(p, *[None] * 7) == BAD
        assert lib.gemm_vocab_loss_run_backward(p, *[None] * 9) == BAD
        assert lib.gemm_vocab_loss_workspace_size(p) == 0
    assert lib.gemm_vocab_loss_plan_destroy(None) == OK
    assert lib.gemm_vocab_loss_plan_destroy(ctypes.addressof(junk)) == BAD
    assert lib.gemm_vocab_loss_plan_create(None, None) == BAD


def storage(rows, cols, pad):
    ld = -(-cols // 8) * 8 + 8 * pad
    full = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    return full, full[:, :cols]


class Loss:
    def __init__(self, T, V, H, seed=0, pad=1, scale=2.0, skip=0.2, train=True):
        g = torch.Generator().manual_seed(seed)
        self.T, self.V, self.H = T, V, H
        _, self.x = storage(T, H, pad)
        _, self.w = storage(V, H, pad)
        self.x.copy_(torch.randn(T, H, generator=g).bfloat16())
        self.w.copy_((torch.randn(V, H, generator=g) * scale / H ** 0.5).bfloat16())
        target = torch.randint(0, V, (T,), generator=g)
        target[torch.rand(T, generator=g) < skip] = -100
        if T > 2:
            target[0], target[1] = 0, V - 1
        self.target = target.cuda()
        self.dloss = (torch.randn(T, generator=g) / T).cuda()
        self.dx_full, self.dx = storage(T, H, pad)
        self.dw_full, self.dw = storage(V, H, pad)
        self.loss = torch.full((T,), float("nan"), device="cuda")
        self.lse = torch.full((T,), float("nan"), device="cuda")
        back = dict(dx_rs=self.dx.stride(0), dw_rs=self.dw.stride(0)) if train else {}
        self.plan = migemm.VocabLossPlan(T, V, H, x_rs=self.x.stride(0), w_rs=self.w.stride(0), **back)
        self.ws = torch.full((self.plan.workspace_size,), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        self.plan.run(self.x, self.w, self.target, self.loss, self.lse, self.ws, stream)

    def backward(self, stream=None):
        self.plan.run_backward(self.x, self.w, self.target, self.lse, self.dloss, self.dx, self.dw,
                               self.ws, stream)

    def check(self, backward=True):
        x, w = self.x.double(), self.w.double()
        counts = (self.target >= 0) & (self.target < self.V)
        at = torch.where(counts, self.target, 0)[:, None]
        logits = x @ w.t()
        size = (x.abs() @ w.abs().t()).amax(1)
        L = (self.H + 4) * U * size
        lse = torch.logsumexp(logits, 1)
        within(self.lse, lse, L + 256 * U + 4 * U * lse.abs())
        picked = logits.gather(1, at).squeeze(1)
        want = torch.where(counts, lse - picked, 0.0)
        within(self.loss, want, torch.where(counts, 2 * L + 256 * U + 6 * U * (lse.abs() + picked.abs()), 0.0))
        if not backward:
            return
        p = torch.softmax(logits, 1)
        dl = torch.where(counts, self.dloss.double(), 0.0)[:, None]
        g = p.clone()
        g[torch.arange(self.T, device="cuda"), at.squeeze(1)] -= 1
        g *= dl
        R = (2 * L + 512 * U + 8 * U * lse.abs())[:, None]
        gerr = R * p * dl.abs() + 2.0 ** -8 * (g.abs() + R * p * dl.abs())
        del p, logits
        for got, ref, mag, err, n in (
                (self.dx, g @ w, g.abs() @ w.abs(), gerr @ w.abs(), self.V),
                (self.dw, g.t().contiguous() @ x, g.abs().t().contiguous() @ x.abs(),
                 gerr.t().contiguous() @ x.abs(), self.T)):
            within(got, ref, err + (n + 8) * U * (mag + err) + 2.0 ** -8 * (ref.abs() + err) + 1e-38)
        assert (self.dx[~counts] == 0).all()
        assert torch.isnan(self.dx_full[:, self.H:].float()).all()
        assert torch.isnan(self.dw_full[:, self.H:].float()).all()


def within(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (over.max().item(), over.argmax().item())


SHAPES = [(1, 1, 1), (1, 100, 64), (1, 5000, 520), (2, 127, 9), (3, 129, 65), (16, 1000, 128),
          (17, 3000, 200), (64, 700, 333), (100, 50000, 200), (130, 127, 72), (257, 300, 136),
          (600, 1000, 40), (1001, 3201, 500), (300, 12000, 1030)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_loss_and_gradients(T, V, H):
    p = Loss(T, V, H, seed=T + V + H)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
def test_rows_in_chunks_and_vocabulary_in_pieces():
    p = Loss(16400, 20000, 24, seed=1)      # 2 launches of rows forward, 2 pieces of g backward
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_flat_and_peaked_logits(scale):
    p = Loss(70, 2000, 96, seed=3, scale=scale)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", [(40, 600, 64), (300, 700, 100)])
def test_masked_rows_reach_nothing(T, V, H):
    """Rows that do not count may hold anything: dx is 0 there and dw is what
    it is with zeros in their place."""
    p, q = Loss(T, V, H, seed=5), Loss(T, V, H, seed=5)
    skip = p.target < 0
    assert skip.any()
    p.x[skip] = float("nan")
    p.dloss[skip] = float("inf")
    for o in (p, q):
        o.forward()
        o.backward()
    torch.cuda.synchronize()
    assert (p.loss[skip] == 0).all() and torch.isnan(p.lse[skip]).all()
    for n in ("dx", "dw"):
        assert torch.equal(getattr(p, n), getattr(q, n)), n
    assert torch.equal(p.loss, q.loss)


@pytest.mark.gpu
def test_no_row_counts():
    p = Loss(50, 300, 40, seed=6)
    p.target.fill_(-1)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    assert (p.loss == 0).all() and (p.dx == 0).all() and (p.dw == 0).all()
    assert torch.isfinite(p.lse).all()


@pytest.mark.gpu
def test_no_rows():
    p = Loss(0, 300, 40)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    assert (p.dw == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 200])
def test_infinite_logits_and_targets_past_the_vocabulary(T):
    p = Loss(T, 400, 8, seed=7, skip=0.0)
    p.x[:] = 1.0
    p.w[:] = 0.0
    p.w[7] = float("-inf")                  # one entry that cannot be chosen
    p.target[0], p.target[1], p.target[2], p.target[3] = 400, 1 << 40, 7, 3
    p.forward()
    torch.cuda.synchronize()
    loss, lse = p.loss.cpu(), p.lse.cpu()
    want = torch.log(torch.tensor(399.0)).item()
    assert (lse - want).abs().max() < 1e-5
    assert torch.isnan(loss[:2]).all() and loss[2] == float("inf") and abs(loss[3] - want) < 1e-5
    p.w[9] = float("inf")
    p.forward()
    torch.cuda.synchronize()
    assert (p.lse == float("inf")).all()
    p.w[:] = float("-inf")
    p.forward()
    torch.cuda.synchronize()
    assert (p.lse == float("-inf")).all()


@pytest.mark.gpu
def test_gradient_against_differences():
    """<dx, u> and <dw, v> against central differences of sum dloss loss in 64
    bits; the bound is test_loss_and_gradients' bound along the direction."""
    p = Loss(33, 500, 48, seed=8)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    x, w = p.x.double(), p.w.double()
    counts = p.target >= 0
    at = torch.where(counts, p.target, 0)[:, None]
    dl = torch.where(counts, p.dloss.double(), 0.0)

    def value(x, w):
        logits = x @ w.t()
        return (dl * (torch.logsumexp(logits, 1) - logits.gather(1, at).squeeze(1))).sum()

    g = torch.softmax(x @ w.t(), 1)
    g[torch.arange(33, device="cuda"), at.squeeze(1)] -= 1
    g = (g * dl[:, None]).abs()
    gen = torch.Generator(device="cuda").manual_seed(2)
    t = 1e-6
    for _ in range(3):
        u = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        v = torch.randn(w.shape, generator=gen, device="cuda", dtype=torch.float64)
        for got, diff, mag in (
                ((p.dx.double() * u).sum(), (value(x + t * u, w) - value(x - t * u, w)) / (2 * t),
                 ((g @ w.abs()) * u.abs()).sum()),
                ((p.dw.double() * v).sum(), (value(x, w + t * v) - value(x, w - t * v)) / (2 * t),
                 ((g.t().contiguous() @ x.abs()) * v.abs()).sum())):
            assert abs(got - diff) <= 2.0 ** -7 * 1.05 * mag


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H", [(5, 3000, 200), (300, 3000, 200)])
def test_runs_agree_on_streams_and_in_a_graph(T, V, H):
    p = Loss(T, V, H, seed=9)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    outs = (p.loss, p.lse, p.dx, p.dw)
    want = [t.clone() for t in outs]

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(a, b) for a, b in zip(want, outs))
        for t in outs:
            t.fill_(7)
        p.ws.fill_(0xFF)
        torch.cuda.synchronize()
        return ok

    assert same()
    s = torch.cuda.Stream()
    p.forward(s)
    p.backward(s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward()
        p.backward()
    for _ in range(3):
        graph.replay()
        assert same()
        p.forward()
        p.backward()
        assert same()


@pytest.mark.gpu
def test_run_refusals():
    p = Loss(4, 40, 64)
    lib, plan, ws = migemm.load(), p.plan.handle, p.ws.data_ptr()
    f = [t.data_ptr() for t in (p.x, p.w, p.target, p.loss, p.lse)]
    b = [t.data_ptr() for t in (p.x, p.w, p.target, p.lse, p.dloss, p.dx, p.dw)]
    for i in range(len(f)):
        assert lib.gemm_vocab_loss_run(plan, *f[:i], None, *f[i + 1:], ws, None) == BAD
        assert lib.gemm_vocab_loss_run(plan, *f[:i], f[i] + 2, *f[i + 1:], ws, None) == MIS
    for i in range(len(b)):
        assert lib.gemm_vocab_loss_run_backward(plan, *b[:i], None, *b[i + 1:], ws, None) == BAD
        assert lib.gemm_vocab_loss_run_backward(plan, *b[:i], b[i] + 2, *b[i + 1:], ws, None) == MIS
    assert lib.gemm_vocab_loss_run(plan, *f, None, None) == BAD
    assert lib.gemm_vocab_loss_run_backward(plan, *b, ws + 16, None) == MIS
    q = Loss(4, 40, 64, train=False)
    assert lib.gemm_vocab_loss_run_backward(q.plan.handle, *b, ws, None) == BAD
    n = migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64)
    assert lib.gemm_vocab_loss_run(n.handle, *f, ws, None) == BAD
