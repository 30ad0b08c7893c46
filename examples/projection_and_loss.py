"""The operators around the product, used together: a residual stream is
normed into 8-bit rows, an 8-bit projection updates it, a second norm makes
bf16 rows, and the loss over a large vocabulary is taken from them without
the logits in memory; then the gradients of the loss, down to the second
norm's input.

    python examples/projection_and_loss.py [--tokens 512] [--hidden 1024] [--vocab 32000]

    r ----------------------------+---------------> h2 --norm--> y2 --vocab loss--> loss
    x --(+ r) h --norm--> e4m3 --scaled product--> p    (h2 = h + p)

Random weights and tokens; one step, checked against the same in fp32.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from warp_specialized_pipelined_amd import migemm  # noqa: E402

EPS = 1e-5


def workspace(plan):
    return torch.empty(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")


class Step:
    """Plans, buffers and weights a program keeps between steps."""

    def __init__(self, tokens, hidden, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*size, scale=1.0):
            return torch.randn(*size, generator=g, device="cuda") * scale

        bf16, fp8 = torch.bfloat16, torch.float8_e4m3fn
        self.w1, self.w2 = (1 + normal(hidden, scale=0.1)).to(bf16), (1 + normal(hidden, scale=0.1)).to(bf16)
        # The projection's weights: e4m3 with a scale per output channel.
        proj = normal(hidden, hidden, scale=hidden ** -0.5)
        self.proj_scale = proj.abs().amax(1) / 448
        self.proj = (proj / self.proj_scale[:, None]).to(fp8)
        self.head = normal(vocab, hidden, scale=2 * hidden ** -0.5).to(bf16)

        def rows(dtype=bf16, n=hidden):
            return torch.empty(tokens, n, dtype=dtype, device="cuda")

        self.h, self.y1, self.p, self.h2, self.y2 = rows(), rows(fp8), rows(), rows(), rows()
        self.scale1 = torch.empty(tokens, device="cuda")
        self.rstd1, self.rstd2 = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.loss, self.lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.dy2, self.dh2 = rows(), rows()
        self.dhead = torch.empty_like(self.head)
        self.dw2 = torch.empty(hidden, device="cuda")

        rs = hidden
        self.norm1 = migemm.NormPlan(tokens, hidden, EPS, migemm.MIGEMM_FP8_E4M3, x_rs=rs, y_rs=rs, r_rs=rs, h_rs=rs)
        self.product = migemm.ScaledPlan(tokens, hidden, hidden, a_rs=rs, b_cs=rs, d_rs=rs)
        self.norm2 = migemm.NormPlan(tokens, hidden, EPS, x_rs=rs, y_rs=rs, r_rs=rs, h_rs=rs, dy_rs=rs, dx_rs=rs)
        self.vocab = migemm.VocabLossPlan(tokens, vocab, hidden, x_rs=rs, w_rs=rs, dx_rs=rs, dw_rs=rs)
        self.ws = {k: workspace(getattr(self, k)) for k in ("product", "norm2", "vocab")}

    def forward(self, x, r, target):
        self.norm1.run(x, r, self.w1, self.h, self.y1, self.scale1, self.rstd1)
        self.product.run(self.y1, self.scale1, self.proj, self.proj_scale, self.p, self.ws["product"])
        self.norm2.run(self.p, self.h, self.w2, self.h2, self.y2, None, self.rstd2)
        self.vocab.run(self.y2, self.head, target, self.loss, self.lse, self.ws["vocab"])
        return self.loss

    def backward(self, target, dloss):
        """Gradients of sum(dloss * loss): the head's, the second norm's
        weight's and those of what the second norm added up."""
        self.vocab.run_backward(self.y2, self.head, target, self.lse, dloss, self.dy2, self.dhead, self.ws["vocab"])
        self.norm2.run_backward(self.dy2, self.h2, self.w2, self.rstd2, None, self.dh2, self.dw2, self.ws["norm2"])
        return self.dhead, self.dw2, self.dh2


def reference(s, x, r, target, dloss):
    """The same in fp32 (the roundings between the operators as theirs)."""
    h = (x.float() + r.float()).bfloat16().float()
    n1 = h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + EPS) * s.w1.float()
    scale = n1.abs().amax(1, keepdim=True) / 448
    q = (n1 / scale).to(torch.float8_e4m3fn).float() * scale
    p = (q @ (s.proj.float() * s.proj_scale[:, None]).t()).bfloat16().float()
    h2 = (p + h).bfloat16().float().requires_grad_()
    w2, head = s.w2.float().requires_grad_(), s.head.float().requires_grad_()
    y2 = (h2 * torch.rsqrt(h2.pow(2).mean(1, keepdim=True) + EPS) * w2)
    loss = torch.nn.functional.cross_entropy(y2 @ head.t(), target, reduction="none", ignore_index=-100)
    (loss * dloss).sum().backward()
    return loss.detach(), head.grad, w2.grad, h2.grad


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args(argv)
    s = Step(a.tokens, a.hidden, a.vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    r = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").mul(2).bfloat16()
    target = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    target[1::10] = -100  # tokens that do not count
    dloss = (target >= 0).float() / (target >= 0).sum()
    loss = s.forward(x, r, target)
    got = (loss, *s.backward(target, dloss))
    want = reference(s, x, r, target, dloss)
    errors = {}
    for name, u, v in zip(("loss", "dhead", "dw2", "dh2"), got, want):
        errors[name] = ((u.float() - v).norm() / v.norm()).item()
    print("mean loss %.4f; relative errors %s" % ((loss * dloss).sum().item(),
                                                 ", ".join("%s %.2g" % e for e in errors.items())))
    return errors


if __name__ == "__main__":
    main()
