"""The operators between and inside the 8-bit products of a block, used together.

    python examples/eight_bit_block.py [--tokens 512] [--hidden 1024] [--wide 4096]

Serving: the block norm makes int8 rows from a block's output, its gate and the
residual, an int8 product with a bias takes them, its result is brought to 8
bits and goes through a second one.

    x, z, r --block norm--> h, int8 rows --int8 product--> a --quantize--> int8 rows --int8 product--> out

Training: the block norm makes bf16 rows, which a product takes and a checkpoint
keeps in 8 bits; the weights' gradient, of two micro-batches, comes from the
kept form and is added up in fp32, and the block norm's backward pass gives those
of the block's output, its gate, the residual and the norms' weights.

Random weights and activations, checked against the same in fp32.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from warp_specialized_pipelined_amd import migemm  # noqa: E402

EPS, BRANCH = 1e-5, 0.5
BF16, INT8, FP32 = migemm.MIGEMM_BF16, migemm.MIGEMM_INT8, migemm.MIGEMM_FP32


def workspace(plan):
    return torch.empty(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")


def rows(tokens, n, dtype=torch.bfloat16):
    return torch.empty(tokens, n, dtype=dtype, device="cuda")


class Inputs:
    def __init__(self, tokens, hidden, wide, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*size, scale=1.0):
            return (torch.randn(*size, generator=g, device="cuda") * scale).bfloat16()

        self.x, self.z, self.r = normal(tokens, hidden), normal(tokens, hidden), normal(tokens, hidden, scale=2.0)
        self.w, self.pw = (1 + normal(hidden, scale=0.1).float()).bfloat16(), (1 + normal(hidden, scale=0.1).float()).bfloat16()
        self.up, self.down = normal(wide, hidden, scale=hidden ** -0.5), normal(hidden, wide, scale=wide ** -0.5)
        self.bias = torch.randn(wide, generator=g, device="cuda")
        self.dp = normal(tokens, wide, scale=0.1)
        self.dh = normal(tokens, hidden, scale=0.1)


def int8_weights(w):
    """Codes with a scale per output channel, by the rows' operator itself."""
    q, scale = rows(*w.shape, dtype=torch.int8), torch.empty(len(w), device="cuda")
    migemm.QuantizePlan(*w.shape, x_rs=w.shape[1], q_rs=w.shape[1]).run(w, q, scale)
    return q, scale


class Serving:
    """Plans, weights and buffers a program keeps between steps."""

    def __init__(self, i):
        (self.tokens, self.hidden), self.wide = i.x.shape, len(i.up)
        t, n, f = self.tokens, self.hidden, self.wide
        self.up, self.down = int8_weights(i.up), int8_weights(i.down)
        self.norm = migemm.BlockNormPlan(t, n, EPS, INT8, branch_scale=BRANCH, x_rs=n, z_rs=n, r_rs=n, h_rs=n, y_rs=n)
        self.first = migemm.Int8Plan(t, f, n, a_rs=n, b_cs=n, d_rs=f)
        self.quantize = migemm.QuantizePlan(t, f, x_rs=f, q_rs=f)
        self.second = migemm.Int8Plan(t, n, f, a_rs=f, b_cs=f, d_rs=n)
        self.h, self.y, self.a, self.q, self.out = rows(t, n), rows(t, n, torch.int8), rows(t, f), rows(t, f, torch.int8), rows(t, n)
        self.scale, self.post_rstd, self.rstd, self.a_scale = (torch.empty(t, device="cuda") for _ in range(4))
        self.ws = workspace(self.first), workspace(self.second)

    def run(self, i, stream=None):
        self.norm.run(i.x, i.z, i.r, i.pw, i.w, self.h, self.y, self.scale, self.post_rstd, self.rstd, stream)
        self.first.run(self.y, self.scale, *self.up, i.bias, self.a, self.ws[0], stream)
        self.quantize.run(self.a, self.q, self.a_scale, stream)
        self.second.run(self.q, self.a_scale, *self.down, None, self.out, self.ws[1], stream)
        return self.h, self.out


class Training:
    def __init__(self, i):
        (t, n), f = i.x.shape, len(i.up)
        names = ("x", "z", "r", "h", "y", "dy", "dh", "dx", "dz", "dr")
        self.norm = migemm.BlockNormPlan(t, n, EPS, branch_scale=BRANCH, **{k + "_rs": n for k in names})
        # p = y up^T, and dy = dp up
        self.product = migemm.Plan(migemm.make_desc(t, f, n, BF16, BF16, n, 1, 1, n, f, 1, f, 1))
        self.back = migemm.Plan(migemm.make_desc(t, n, f, BF16, BF16, f, 1, n, 1, n, 1, n, 1))
        self.checkpoint = migemm.CheckpointPlan(t, n, x_rs=n, out_cols=f, dy_rs=f, dw_rs=n, dw_type=FP32, accumulate=True)
        self.kept = torch.empty(max(self.checkpoint.checkpoint_size, 16), dtype=torch.uint8, device="cuda")
        self.h, self.y, self.p, self.dy = rows(t, n), rows(t, n), rows(t, f), rows(t, n)
        self.dx, self.dz, self.dr = rows(t, n), rows(t, n), rows(t, n)
        self.post_rstd, self.rstd = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        self.dw, self.dpw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        self.dup = torch.zeros(f, n, device="cuda")
        self.ws = workspace(self.norm), workspace(self.checkpoint)

    def forward(self, i, stream=None):
        self.norm.run(i.x, i.z, i.r, i.pw, i.w, self.h, self.y, None, self.post_rstd, self.rstd, stream)
        self.checkpoint.pack(self.y, self.kept, stream)
        self.product.run(self.y, i.up, None, self.p, stream=stream)
        return self.p

    def backward(self, i, stream=None):
        """y itself is not read: what it was is in the kept form."""
        self.checkpoint.weight_gradient(i.dp, self.kept, self.dup, self.ws[1], stream)
        self.back.run(i.dp, i.up, None, self.dy, stream=stream)
        self.norm.run_backward(self.dy, i.dh, i.x, i.z, self.h, i.pw, i.w, self.post_rstd, self.rstd, self.dx, self.dz,
                               self.dr, self.dpw, self.dw, self.ws[0], stream)


def block(x, z, r, pw, w):
    u = x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + EPS) * pw
    h = r + BRANCH * torch.sigmoid(z) * u
    return h, h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + EPS) * w


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--wide", type=int, default=4096)
    a = ap.parse_args(argv)
    batches = [Inputs(a.tokens, a.hidden, a.wide, seed) for seed in (1, 2)]
    batches[1].up, batches[1].w, batches[1].pw = batches[0].up, batches[0].w, batches[0].pw
    i = batches[0]
    errors = {}

    def off(name, got, want):
        errors[name] = ((got.float() - want).norm() / want.norm()).item()

    serving = Serving(i)
    h, out = serving.run(i)
    h32, y32 = block(*(t.float() for t in (i.x, i.z, i.r, i.pw, i.w)))
    off("h", h, h32)
    off("out", out, (y32 @ i.up.float().t() + i.bias) @ i.down.float().t())

    training = Training(i)
    want_up, kept_up = 0.0, 0.0
    for b in batches:
        training.forward(b)
        training.backward(b)
        leaves = [t.float().requires_grad_() for t in (b.x, b.z, b.r, b.pw, b.w)]
        h32, y32 = block(*leaves)
        ((y32 @ b.up.float().t()) * b.dp.float()).sum().add((h32 * b.dh.float()).sum()).backward()
        y_kept = torch.empty_like(training.y)
        training.checkpoint.unpack(training.kept, y_kept)
        want_up, kept_up = want_up + b.dp.float().t() @ y32.detach(), kept_up + b.dp.float().t() @ y_kept.float()
    off("p", training.p, y32.detach() @ b.up.float().t())
    for name, got, t in zip(("dx", "dz", "dr", "dpost_weight", "dweight"),
                            (training.dx, training.dz, training.dr, training.dpw, training.dw), leaves):
        off(name, got, t.grad)
    off("dup_kept", training.dup, kept_up)
    off("dup", training.dup, want_up)
    print("relative errors " + ", ".join("%s %.2g" % e for e in errors.items()))
    return errors


if __name__ == "__main__":
    main()
