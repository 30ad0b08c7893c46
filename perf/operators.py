"""The operators around a product, at the sizes they are measured at.

Three operators that stand on either side of the library's GEMM in a large
language model, each as a user's program calls it:

  norm    the residual's addition and the root-mean-square norm of each row;
          the result in bf16 (training) or in e4m3 with a scale per row (the
          operand of the 8-bit product), and its gradient;
  scaled  the 8-bit product: e4m3 rows with a scale each times e4m3 weights
          with a scale per output channel, from one token to long prompts;
  loss    softmax cross entropy over a large vocabulary from the hidden states
          and the output projection's weights, without the logits in memory,
          and the gradients of both.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, with the library.  ``exact`` gives the same outputs in 64
bits, from the definitions alone.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
IGNORED = -100


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One token's hidden state between two 8-bit projections: all latency.
        {"name": "norm_one_token_e4m3", "op": "norm", "step": "forward", "rows": 1, "cols": 8192,
         "out": "e4m3", "residual": True},
        # A long prompt in front of an 8-bit projection.
        {"name": "norm_prompt_e4m3", "op": "norm", "step": "forward", "rows": 8192, "cols": 8192,
         "out": "e4m3", "residual": True},
        # The first norm of a stack (nothing to add yet), sizes of no power of two.
        {"name": "norm_ragged_bf16", "op": "norm", "step": "forward", "rows": 4000, "cols": 5000,
         "out": "bf16", "residual": False},
        # A training step's norm: forward, then the gradients of the input and the weight.
        {"name": "norm_train", "op": "norm", "step": "train", "rows": 8192, "cols": 4096,
         "out": "bf16", "residual": True},
        # One token through a square projection: the weights' bytes decide.
        {"name": "scaled_one_token", "op": "scaled", "rows": 1, "cols": 8192, "inner": 8192},
        # A batch of single tokens through a wide projection.
        {"name": "scaled_batch_40", "op": "scaled", "rows": 40, "cols": 16384, "inner": 8192},
        # A prompt of ragged sizes, none a multiple of a tile.
        {"name": "scaled_ragged", "op": "scaled", "rows": 4000, "cols": 3000, "inner": 5000},
        # A long prompt: matrix instructions decide.
        {"name": "scaled_prompt", "op": "scaled", "rows": 8192, "cols": 8192, "inner": 16384},
        # Scoring one short answer of a small model.
        {"name": "loss_score_short", "op": "loss", "step": "forward", "rows": 100, "vocab": 50000,
         "hidden": 1000},
        # Evaluation of a batch over a large vocabulary.
        {"name": "loss_evaluate", "op": "loss", "step": "forward", "rows": 4096, "vocab": 131072,
         "hidden": 4096},
        # A small training step, odd tokens and an odd vocabulary.
        {"name": "loss_train_ragged", "op": "loss", "step": "train", "rows": 1001, "vocab": 32001,
         "hidden": 2000},
        # A large training step: 8192 tokens, 131072 entries.
        {"name": "loss_train", "op": "loss", "step": "train", "rows": 8192, "vocab": 131072,
         "hidden": 4096},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "scaled", "loss"])
    if op == "norm":
        return {"op": "norm", "step": rng.choice(["forward", "forward", "train"]),
                "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 64, 8192),
                "out": rng.choice(["bf16", "e4m3"]), "residual": rng.choice([True, True, False])}
    if op == "scaled":
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
        return {"op": "scaled", "rows": rows, "cols": cols, "inner": _spread(rng, 64, 16384)}
    return {"op": "loss", "step": rng.choice(["forward", "train"]), "rows": _spread(rng, 1, 8192),
            "vocab": _spread(rng, 100, 131072), "hidden": _spread(rng, 64, 4096)}


def work(case):
    if case["op"] == "norm":
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        # x, and the residual in and out where there is one
        b = n * (2 + (4 if case["residual"] else 0)) + 2 * cols + 4 * rows
        if case["step"] == "train":  # y; dy, and the residual's gradient; dx, dweight
            b += n * (2 + 2 + (2 if case["residual"] else 0) + 2) + 4 * cols
            return {"bytes": b, "flops": 14 * n}
        b += n * 2 if case["out"] == "bf16" else n + 4 * rows
        return {"bytes": b, "flops": 5 * n}
    if case["op"] == "scaled":
        m, n, k = case["rows"], case["cols"], case["inner"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n, "flops": 2 * m * n * k}
    t, v, h = case["rows"], case["vocab"], case["hidden"]
    b, f = 2 * h * (t + v) + 8 * t + 8 * t, 2 * t * v * h
    if case["step"] == "train":  # both gradients, and two more products of the same size
        b, f = b + 2 * h * (t + v) + 4 * t, 3 * f
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------- the inputs

def _padded(rows, cols, dtype):
    """A rows x cols matrix whose rows start at multiples of 16 bytes, as the library wants them."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = -(-cols // per) * per
    return torch.empty((rows, ld), dtype=dtype, device=DEVICE)[:, :cols]


def _normal(gen, rows, cols, scale=1.0, column=None):
    m = _padded(rows, cols, torch.bfloat16)
    v = torch.randn((rows, cols), generator=gen, device=DEVICE)
    if column is not None:
        v *= column
    m.copy_(v * scale)
    return m


def _codes(gen, rows, cols):
    """Rows of N(0, 1) in e4m3 with a scale each (the row's largest magnitude is 448)."""
    v = torch.randn((rows, cols), generator=gen, device=DEVICE)
    scale = v.abs().amax(1) / E4M3_MAX
    q = _padded(rows, cols, torch.float8_e4m3fn)
    q.copy_((v / scale[:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
    return q, scale


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # A residual stream with a few large channels, as trained models have.
        column = 1 + 20 * (torch.rand(cols, generator=gen, device=DEVICE) < 0.003)
        s = {"x": _normal(gen, rows, cols)}
        if case["residual"]:
            s["r"] = _normal(gen, rows, cols, 2.0, column)
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=DEVICE)).bfloat16()
        if case["step"] == "train":
            s["dy"] = _normal(gen, rows, cols, 0.01)
            if case["residual"]:
                s["dh"] = _normal(gen, rows, cols, 0.01)
        return s
    if case["op"] == "scaled":
        a, a_scale = _codes(gen, case["rows"], case["inner"])
        b, b_scale = _codes(gen, case["cols"], case["inner"])
        return {"a": a, "a_scale": a_scale, "b": b, "b_scale": b_scale / math.sqrt(case["inner"])}
    t, v, h = case["rows"], case["vocab"], case["hidden"]
    # Normed hidden states, weights that give logits of about N(0, 2^2); one
    # token in ten (a prompt's, or padding) does not count.
    s = {"x": _normal(gen, t, h), "w": _normal(gen, v, h, 2.0 / math.sqrt(h))}
    target = torch.randint(0, v, (t,), generator=gen, device=DEVICE)
    skip = torch.rand(t, generator=gen, device=DEVICE) < 0.1
    skip[0] = False
    s["target"] = torch.where(skip, IGNORED, target)
    counts = s["target"] >= 0
    s["dloss"] = counts.float() / counts.sum()  # the mean over the tokens that count
    return s


def prepare(case, seed):
    state = {"case": dict(case), **_inputs(case, seed)}
    if own:
        _plan(case, state)
    return state


def _plan(case, s):
    """What a user of the library keeps: the plan, its workspace and the output buffers."""
    from warp_specialized_pipelined_amd import migemm
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        train, e4m3 = case["step"] == "train", case["out"] == "e4m3" and case["step"] != "train"
        y = _padded(rows, cols, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        h = _padded(rows, cols, torch.bfloat16) if case["residual"] else None
        s["y"], s["h"] = y, h
        s["rstd"] = torch.empty(rows, device=DEVICE)
        s["scale"] = torch.empty(rows, device=DEVICE) if e4m3 else None
        strides = {"x_rs": s["x"].stride(0), "y_rs": y.stride(0)}
        if h is not None:
            strides.update(r_rs=s["r"].stride(0), h_rs=h.stride(0))
        if train:
            s["dx"] = _padded(rows, cols, torch.bfloat16)
            s["dweight"] = torch.empty(cols, device=DEVICE)
            strides.update(dy_rs=s["dy"].stride(0), dx_rs=s["dx"].stride(0))
            if h is not None:
                strides.update(dh_rs=s["dh"].stride(0))
        s["plan"] = migemm.NormPlan(rows, cols, EPS,
                                    migemm.MIGEMM_FP8_E4M3 if e4m3 else migemm.MIGEMM_BF16,
                                    **strides)
    elif case["op"] == "scaled":
        s["d"] = _padded(case["rows"], case["cols"], torch.bfloat16)
        s["plan"] = migemm.ScaledPlan(case["rows"], case["cols"], case["inner"],
                                      a_rs=s["a"].stride(0), b_cs=s["b"].stride(0),
                                      d_rs=s["d"].stride(0))
    else:
        t, v, h = case["rows"], case["vocab"], case["hidden"]
        strides = {"x_rs": s["x"].stride(0), "w_rs": s["w"].stride(0)}
        s["loss"], s["lse"] = torch.empty(t, device=DEVICE), torch.empty(t, device=DEVICE)
        if case["step"] == "train":
            s["dx"], s["dw"] = _padded(t, h, torch.bfloat16), _padded(v, h, torch.bfloat16)
            strides.update(dx_rs=s["dx"].stride(0), dw_rs=s["dw"].stride(0))
        s["plan"] = migemm.VocabLossPlan(t, v, h, **strides)
    size = s["plan"].workspace_size
    s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEVICE) if size else None


# ----------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        return _norm(case, state)
    if case["op"] == "scaled":
        return _scaled(state)
    return _loss(case, state)


def _run_own(case, s):
    plan = s["plan"]
    if case["op"] == "norm":
        plan.run(s["x"], s.get("r"), s["weight"], s["h"], s["y"], s["scale"], s["rstd"])
        out = {"y": s["y"], "rstd": s["rstd"]}
        if s["h"] is not None:
            out["h"] = s["h"]
        if s["scale"] is not None:
            out["scale"] = s["scale"]
        if case["step"] == "train":
            plan.run_backward(s["dy"], s["h"] if s["h"] is not None else s["x"], s["weight"],
                              s["rstd"], s.get("dh"), s["dx"], s["dweight"], s["workspace"])
            out.update(dx=s["dx"], dweight=s["dweight"])
        return out
    if case["op"] == "scaled":
        plan.run(s["a"], s["a_scale"], s["b"], s["b_scale"], s["d"], s["workspace"])
        return {"d": s["d"]}
    plan.run(s["x"], s["w"], s["target"], s["loss"], s["lse"], s["workspace"])
    out = {"loss": s["loss"], "lse": s["lse"]}
    if case["step"] == "train":
        plan.run_backward(s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dx"], s["dw"],
                          s["workspace"])
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def _norm(case, s):
    if case["residual"]:
        h = (s["x"].float() + s["r"].float()).bfloat16()
    else:
        h = s["x"]
    hf, w = h.float(), s["weight"].float()
    rstd = torch.rsqrt((hf * hf).mean(1) + EPS)
    normed = hf * rstd[:, None]
    y = normed * w
    out = {"rstd": rstd}
    if case["residual"]:
        out["h"] = h
    if case["step"] == "train":
        g = s["dy"].float()
        gw = g * w
        d = rstd[:, None] * (gw - normed * (gw * normed).mean(1, keepdim=True))
        if case["residual"]:
            d = d + s["dh"].float()
        out.update(y=y.bfloat16(), dx=d.bfloat16(), dweight=(g * normed).sum(0))
    elif case["out"] == "bf16":
        out["y"] = y.bfloat16()
    else:
        largest = y.abs().amax(1)
        scale = largest / E4M3_MAX
        q = y * torch.where(largest > 0, E4M3_MAX / largest, 0.0)[:, None]
        out.update(scale=scale, y=q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
    return out


def _scaled(s):
    d = s["a"].float() @ s["b"].float().t()
    return {"d": (d * s["a_scale"][:, None] * s["b_scale"]).bfloat16()}


def _loss(case, s):
    x, w = s["x"].float(), s["w"].float()
    logits = x @ w.t()
    largest = logits.amax(1, keepdim=True)
    lse = (largest + (logits - largest).exp().sum(1, keepdim=True).log()).squeeze(1)
    counts = s["target"] >= 0
    at = s["target"].clamp(min=0)[:, None]
    loss = torch.where(counts, lse - logits.gather(1, at).squeeze(1), 0.0)
    out = {"loss": loss, "lse": lse}
    if case["step"] == "train":
        g = (logits - lse[:, None]).exp()
        g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        g *= torch.where(counts, s["dloss"], 0.0)[:, None]
        out.update(dx=(g @ w).bfloat16(), dw=(g.t() @ x).bfloat16())
    return out


# ------------------------------------------------------ the same in 64 bits

def _e4m3_grid(v):
    """The nearest e4m3 values (ties to even): 3 bits of fraction, exponents from -6 on."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        h = s["x"]
        if case["residual"]:
            h = (s["x"].double() + s["r"].double()).to(torch.bfloat16)
        rows, cols = case["rows"], case["cols"]
        w = s["weight"].double()
        out = {k: [] for k in ("rstd", "y", "scale", "dx")}
        dweight = torch.zeros(cols, dtype=torch.float64, device=DEVICE)
        for a in range(0, rows, 1024):
            v = h[a:a + 1024].double()
            norm = (v.pow(2).sum(1) / cols + EPS).pow(0.5)
            n = v / norm[:, None]
            out["rstd"].append(1 / norm)
            if case["step"] == "train":
                out["y"].append(n * w)
                g = s["dy"][a:a + 1024].double()
                inner = (g * w * n).sum(1, keepdim=True) / cols
                d = (g * w - inner * n) / norm[:, None]
                if case["residual"]:
                    d += s["dh"][a:a + 1024].double()
                out["dx"].append(d)
                dweight += (g * n).sum(0)
            elif case["out"] == "bf16":
                out["y"].append(n * w)
            else:
                top = (n * w).abs().max(1).values
                out["scale"].append(top / E4M3_MAX)
                out["y"].append(_e4m3_grid(n * w / torch.where(top > 0, top, 1.0)[:, None] * E4M3_MAX))
        got = {k: torch.cat(v) for k, v in out.items() if v}
        if case["residual"]:
            got["h"] = h.double()
        if case["step"] == "train":
            got["dweight"] = dweight
        return got
    if case["op"] == "scaled":
        b = s["b"].double() * s["b_scale"].double()[:, None]
        return {"d": torch.mm(s["a"].double() * s["a_scale"].double()[:, None], b.t())}
    t, v, h = case["rows"], case["vocab"], case["hidden"]
    train, w = case["step"] == "train", s["w"].double()
    loss = torch.zeros(t, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(t, dtype=torch.float64, device=DEVICE)
    dx = torch.zeros((t, h), dtype=torch.float64, device=DEVICE)
    dw = torch.zeros((v, h), dtype=torch.float64, device=DEVICE) if train else None
    for a in range(0, t, 1024):
        x = s["x"][a:a + 1024].double()
        logits = torch.mm(x, w.t())
        lse[a:a + 1024] = torch.logsumexp(logits, 1)
        rows = (s["target"][a:a + 1024] >= 0).nonzero().squeeze(1)
        target = s["target"][a:a + 1024][rows]
        loss[a + rows] = lse[a + rows] - logits[rows, target]
        if train:
            p = torch.softmax(logits[rows], 1)
            p[torch.arange(len(rows), device=DEVICE), target] -= 1
            p *= s["dloss"][a + rows].double()[:, None]
            dx[a + rows] = torch.mm(p, w)
            dw += torch.mm(p.t().contiguous(), x[rows])
    got = {"loss": loss, "lse": lse}
    if train:
        got.update(dx=dx, dw=dw)
    return got
