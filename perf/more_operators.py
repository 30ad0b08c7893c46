"""More operators around a product, at the sizes they are measured at.

Four operators that belong to a block of a large language model whose products
run in 8 bits, or whose activations are kept in 8 bits for the backward pass,
each as a user's program calls it:

  int8        the product of int8 rows with a scale each and int8 weights with
              a scale per output channel, with or without a bias;
  quantize    bf16 rows to int8 or e4m3 with a scale each: what the 8-bit
              products take where no norm stands in front of them;
  block_norm  what stands between two blocks: the norm of a block's output, its
              gate and scale, the residual's addition and the next block's
              norm, in one pass, and the gradients;
  checkpoint  activations kept in 8 bits for the backward pass (e4m3, a power
              of two for each column of 32 tokens), and the weights' gradient
              from them.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, with the library.  ``exact`` gives the same outputs in 64
bits, from the definitions alone.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
TOP = {"int8": 127.0, "e4m3": 448.0}
E4M3 = torch.float8_e4m3fn
BRANCH, RESIDUAL = 0.25, 1.0  # block_norm's scales of the branch and of the residual


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One token through a square projection: the weights' bytes decide.
        {"name": "int8_one_token", "op": "int8", "rows": 1, "cols": 8192, "inner": 8192, "bias": False},
        # A batch of single tokens, an odd number of them, through a wide projection with a bias.
        {"name": "int8_batch_33", "op": "int8", "rows": 33, "cols": 16384, "inner": 8192, "bias": True},
        # A prompt of ragged sizes, none a multiple of a tile.
        {"name": "int8_ragged", "op": "int8", "rows": 4000, "cols": 3000, "inner": 5000, "bias": True},
        # A long prompt: matrix instructions decide.
        {"name": "int8_prompt", "op": "int8", "rows": 8192, "cols": 8192, "inner": 16384, "bias": False},
        # The activations of a batch of single tokens in front of a down projection.
        {"name": "quantize_batch_33", "op": "quantize", "rows": 33, "cols": 8192, "out": "int8"},
        # Those of a long prompt.
        {"name": "quantize_prompt", "op": "quantize", "rows": 8192, "cols": 16384, "out": "int8"},
        # One token between two blocks, in front of an 8-bit projection: all latency.
        {"name": "block_norm_one_token_e4m3", "op": "block_norm", "step": "forward", "rows": 1, "cols": 8192,
         "out": "e4m3", "post": True, "gate": False},
        # A long prompt between two gated blocks, in front of an 8-bit projection.
        {"name": "block_norm_prompt_e4m3", "op": "block_norm", "step": "forward", "rows": 8192, "cols": 8192,
         "out": "e4m3", "post": True, "gate": True},
        # The backward pass of a training step between two gated blocks.
        {"name": "block_norm_backward", "op": "block_norm", "step": "backward", "rows": 8192, "cols": 4096,
         "out": "bf16", "post": True, "gate": True},
        # A training step keeps a projection's input.
        {"name": "checkpoint_pack", "op": "checkpoint", "step": "pack", "rows": 8192, "cols": 8192},
        # The weights' gradient of a small projection, odd tokens and sizes.
        {"name": "checkpoint_gradient_ragged", "op": "checkpoint", "step": "gradient", "rows": 1001, "cols": 2000,
         "out_cols": 5000, "out": "bf16"},
        # That of a large one, into fp32 gradients.
        {"name": "checkpoint_gradient", "op": "checkpoint", "step": "gradient", "rows": 8192, "cols": 8192,
         "out_cols": 8192, "out": "fp32"},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["int8", "int8", "quantize", "block_norm", "block_norm", "checkpoint", "checkpoint"])
    if op == "int8":
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
        return {"op": op, "rows": rows, "cols": cols, "inner": _spread(rng, 64, 16384),
                "bias": rng.choice([True, False])}
    if op == "quantize":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 64, 16384),
                "out": rng.choice(["int8", "int8", "e4m3"])}
    if op == "block_norm":
        step = rng.choice(["forward", "backward"])
        return {"op": op, "step": step, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 64, 8192),
                "out": rng.choice(["bf16", "e4m3"]) if step == "forward" else "bf16",
                "post": rng.choice([True, True, False]), "gate": rng.choice([True, False])}
    rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
    if rng.random() < 0.3:
        return {"op": op, "step": "pack", "rows": rows, "cols": cols}
    return {"op": op, "step": "gradient", "rows": rows, "cols": cols, "out_cols": _spread(rng, 64, 8192),
            "out": rng.choice(["bf16", "fp32"])}


def _up(v, to):
    return -(-v // to) * to


def work(case):
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "int8":
        k = case["inner"]
        b = rows * k + cols * k + 4 * (rows + cols) + 2 * n + (4 * cols if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * n * k}
    if case["op"] == "quantize":
        return {"bytes": 3 * n + 4 * rows, "flops": 4 * n}
    if case["op"] == "block_norm":
        weights = 2 * cols * (2 if case["post"] else 1)
        rstds = 4 * rows * (2 if case["post"] else 1)
        gate = 2 * n if case["gate"] else 0
        if case["step"] == "forward":  # x, r, h; the gate; y
            y = n + 4 * rows if case["out"] == "e4m3" else 2 * n
            return {"bytes": 6 * n + gate + y + weights + rstds, "flops": 14 * n}
        # dy, dh, x, h; dx, dr; the gate and its gradient; the weights' gradients
        return {"bytes": 12 * n + 2 * gate + 3 * weights + rstds, "flops": 30 * n}
    kept = n + n // 32
    if case["step"] == "pack":
        return {"bytes": 2 * n + kept, "flops": 2 * n}
    o = case["out_cols"]
    return {"bytes": kept + 2 * rows * o + (2 if case["out"] == "bf16" else 4) * cols * o, "flops": 2 * n * o}


# --------------------------------------------------------------- the inputs

def _padded(rows, cols, dtype):
    """A rows x cols matrix whose rows start at multiples of 16 bytes, as the library wants them."""
    ld = _up(cols, 16 // torch.empty((), dtype=dtype).element_size())
    return torch.empty((rows, ld), dtype=dtype, device=DEVICE)[:, :cols]


def _normal(gen, rows, cols, scale=1.0, column=None):
    m = _padded(rows, cols, torch.bfloat16)
    v = torch.randn((rows, cols), generator=gen, device=DEVICE)
    if column is not None:
        v *= column
    m.copy_(v * scale)
    return m


def _outliers(gen, cols):
    """A few large channels, as the activations of trained models have."""
    return 1 + 20 * (torch.rand(cols, generator=gen, device=DEVICE) < 0.003)


def _codes(gen, rows, cols, column=None):
    """Rows of N(0, 1) (times `column`) in int8 with a scale each."""
    v = torch.randn((rows, cols), generator=gen, device=DEVICE)
    if column is not None:
        v *= column
    scale = v.abs().amax(1) / 127
    q = _padded(rows, cols, torch.int8)
    q.copy_((v / scale[:, None]).round_().clamp_(-127, 127))
    return q, scale


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "int8":
        k = case["inner"]
        a, a_scale = _codes(gen, rows, k, _outliers(gen, k))
        b, b_scale = _codes(gen, cols, k)
        s = {"a": a, "a_scale": a_scale, "b": b, "b_scale": b_scale / math.sqrt(k)}
        if case["bias"]:
            s["bias"] = torch.randn(cols, generator=gen, device=DEVICE)
        return s
    if case["op"] == "quantize":
        # What an activation function leaves: a product of two normal values.
        return {"x": _normal(gen, rows, cols, 1.0, torch.randn((rows, cols), generator=gen, device=DEVICE))}
    if case["op"] == "block_norm":
        s = {"x": _normal(gen, rows, cols), "r": _normal(gen, rows, cols, 2.0, _outliers(gen, cols)),
             "weight": (1 + 0.2 * torch.randn(cols, generator=gen, device=DEVICE)).bfloat16()}
        if case["post"]:
            s["post_weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=DEVICE)).bfloat16()
        if case["gate"]:
            s["z"] = _normal(gen, rows, cols)
        if case["step"] == "backward":  # what the forward pass left, and the gradients that come in
            f = _block_norm({**case, "out": "bf16"}, s)
            s["h"] = _padded(rows, cols, torch.bfloat16)
            s["h"].copy_(f["h"])
            s["rstd"] = f["rstd"]
            if case["post"]:
                s["post_rstd"] = f["post_rstd"]
            s["dy"], s["dh"] = _normal(gen, rows, cols, 0.01), _normal(gen, rows, cols, 0.01)
        return s
    x = _normal(gen, rows, cols, 1.0, _outliers(gen, cols))
    if case["step"] == "pack":
        return {"x": x}
    kept = _pack(x)
    return {"kept": torch.cat([kept["codes"].view(torch.uint8).flatten(), kept["scales"].flatten()]),
            "dy": _normal(gen, rows, case["out_cols"], 0.01)}


def prepare(case, seed):
    state = {"case": dict(case), **_inputs(case, seed)}
    if own:
        _plan(case, state)
    return state


def _plan(case, s):
    """What a user of the library keeps: the plan, its workspace and the output buffers."""
    from warp_specialized_pipelined_amd import migemm
    rows, cols = case["rows"], case["cols"]
    kinds = {"bf16": migemm.MIGEMM_BF16, "e4m3": migemm.MIGEMM_FP8_E4M3, "int8": migemm.MIGEMM_INT8,
             "fp32": migemm.MIGEMM_FP32}
    types = {"bf16": torch.bfloat16, "e4m3": E4M3, "int8": torch.int8, "fp32": torch.float32}
    if case["op"] == "int8":
        s["d"] = _padded(rows, cols, torch.bfloat16)
        s["plan"] = migemm.Int8Plan(rows, cols, case["inner"], a_rs=s["a"].stride(0), b_cs=s["b"].stride(0),
                                    d_rs=s["d"].stride(0))
    elif case["op"] == "quantize":
        s["q"], s["scale"] = _padded(rows, cols, types[case["out"]]), torch.empty(rows, device=DEVICE)
        s["plan"] = migemm.QuantizePlan(rows, cols, kinds[case["out"]], x_rs=s["x"].stride(0),
                                        q_rs=s["q"].stride(0))
        return
    elif case["op"] == "block_norm":
        strides = {"x_rs": s["x"].stride(0)}
        if case["gate"]:
            strides["z_rs"] = s["z"].stride(0)
        names = ["h"] if case["step"] == "forward" else ["dx", "dr"] + (["dz"] if case["gate"] else [])
        for n in names:
            s[n] = _padded(rows, cols, torch.bfloat16)
        s["y"] = _padded(rows, cols, types[case["out"]])
        s["scale"] = torch.empty(rows, device=DEVICE) if case["out"] != "bf16" else None
        if case["step"] == "forward":
            s["rstd"] = torch.empty(rows, device=DEVICE)
            s["post_rstd"] = torch.empty(rows, device=DEVICE) if case["post"] else None
        else:
            s["dweight"] = torch.empty(cols, device=DEVICE)
            s["dpost_weight"] = torch.empty(cols, device=DEVICE) if case["post"] else None
            strides.update({n + "_rs": s[n].stride(0) for n in ["dy", "dh"] + names})
        s["plan"] = migemm.BlockNormPlan(rows, cols, EPS, kinds[case["out"]], post_norm=case["post"],
                                         branch_scale=BRANCH, residual_scale=RESIDUAL, r_rs=s["r"].stride(0),
                                         h_rs=s["h"].stride(0), y_rs=s["y"].stride(0), **strides)
    elif case["step"] == "pack":
        s["plan"] = migemm.CheckpointPlan(rows, cols, x_rs=s["x"].stride(0))
        s["kept"] = torch.empty(s["plan"].checkpoint_size, dtype=torch.uint8, device=DEVICE)
    else:
        o = case["out_cols"]
        s["dw"] = _padded(o, cols, types[case["out"]])
        s["plan"] = migemm.CheckpointPlan(rows, cols, x_rs=_up(cols, 8), out_cols=o, dy_rs=s["dy"].stride(0),
                                          dw_rs=s["dw"].stride(0), dw_type=kinds[case["out"]])
    size = s["plan"].workspace_size
    s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEVICE) if size else None


# ----------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "int8":
        return _int8(state)
    if case["op"] == "quantize":
        return _quantize(case, state)
    if case["op"] == "block_norm":
        return _block_norm(case, state) if case["step"] == "forward" else _block_norm_backward(case, state)
    return _pack(state["x"]) if case["step"] == "pack" else _gradient(case, state)


def _run_own(case, s):
    plan = s["plan"]
    if case["op"] == "int8":
        plan.run(s["a"], s["a_scale"], s["b"], s["b_scale"], s.get("bias"), s["d"], s["workspace"])
        return {"d": s["d"]}
    if case["op"] == "quantize":
        plan.run(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if case["op"] == "block_norm":
        if case["step"] == "forward":
            plan.run(s["x"], s.get("z"), s["r"], s.get("post_weight"), s["weight"], s["h"], s["y"], s["scale"],
                     s["post_rstd"], s["rstd"])
            names = ["h", "y", "rstd"] + (["scale"] if s["scale"] is not None else [])
            return {n: s[n] for n in names + (["post_rstd"] if case["post"] else [])}
        plan.run_backward(s["dy"], s["dh"], s["x"], s.get("z"), s["h"], s.get("post_weight"), s["weight"],
                          s.get("post_rstd"), s["rstd"], s["dx"], s.get("dz"), s["dr"], s["dpost_weight"],
                          s["dweight"], s["workspace"])
        names = ["dx", "dr", "dweight"] + (["dz"] if case["gate"] else []) + (["dpost_weight"] if case["post"] else [])
        return {n: s[n] for n in names}
    if case["step"] == "pack":
        plan.pack(s["x"], s["kept"])
        n = plan.info.code_bytes
        return {"codes": s["kept"][:n].view(E4M3), "scales": s["kept"][n:]}
    plan.weight_gradient(s["dy"], s["kept"], s["dw"], s["workspace"])
    return {"dw": s["dw"]}


def _int8(s):
    d = (s["a"].float() @ s["b"].float().t()) * s["a_scale"][:, None] * s["b_scale"]
    if "bias" in s:
        d = d + s["bias"]
    return {"d": d.bfloat16()}


def _quantize(case, s):
    top = TOP[case["out"]]
    largest = s["x"].abs().amax(1).float()
    # (64 bits: a quotient on the border of two codes is one exactly.)
    v = s["x"].double() * top / torch.where(largest > 0, largest, 1.0).double()[:, None]
    if case["out"] == "int8":
        return {"q": v.round().to(torch.int8), "scale": largest / top}
    return {"q": v.float().to(E4M3), "scale": largest / top}


def _block_norm(case, s):
    x, w = s["x"].float(), s["weight"].float()
    out = {}
    if case["post"]:
        out["post_rstd"] = torch.rsqrt((x * x).mean(1) + EPS)
        x = x * out["post_rstd"][:, None] * s["post_weight"].float()
    if case["gate"]:
        x = x * torch.sigmoid(s["z"].float())
    h = RESIDUAL * s["r"].float() + BRANCH * x
    out["h"] = h.bfloat16()
    out["rstd"] = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * out["rstd"][:, None] * w
    if case["out"] == "bf16":
        out["y"] = y.bfloat16()
    else:
        largest = y.abs().amax(1)
        out["scale"] = largest / TOP["e4m3"]
        q = y * torch.where(largest > 0, TOP["e4m3"] / largest, 0.0)[:, None]
        out["y"] = q.clamp(-TOP["e4m3"], TOP["e4m3"]).to(E4M3)
    return out


def _block_norm_backward(case, s):
    x, h, w, g = s["x"].float(), s["h"].float(), s["weight"].float(), s["dy"].float()
    out = {}
    n = h * s["rstd"][:, None]
    out["dweight"] = (g * n).sum(0)
    gw = g * w
    dh = s["dh"].float() + s["rstd"][:, None] * (gw - n * (gw * n).mean(1, keepdim=True))
    out["dr"] = (RESIDUAL * dh).bfloat16()
    du = BRANCH * dh
    p = x * s["post_rstd"][:, None] if case["post"] else x
    u = p * s["post_weight"].float() if case["post"] else x
    if case["gate"]:
        gate = torch.sigmoid(s["z"].float())
        out["dz"] = (du * u * gate * (1 - gate)).bfloat16()
        du = du * gate
    if case["post"]:
        out["dpost_weight"] = (du * p).sum(0)
        dp = du * s["post_weight"].float()
        du = s["post_rstd"][:, None] * (dp - p * (dp * p).mean(1, keepdim=True))
    out["dx"] = du.bfloat16()
    return out


def _pack(x):
    """codes [groups of 16 tokens][columns, padded to 16][16 tokens] in e4m3, and for each 32 tokens of a column the
    exponent of its power of two, plus 127."""
    rows, cols = x.shape
    v = torch.zeros((_up(rows, 32), _up(cols, 16)), device=x.device)
    v[:rows, :cols] = x
    v = v.view(-1, 32, v.shape[1])
    fraction, e = torch.frexp(v.abs().amax(1))  # fraction in [1/2, 1)
    e = torch.where(fraction > 0, e + 118 + (fraction > 0.875).int(), 0).clamp(18, 246)
    scale = (e << 23).int().view(torch.float32)
    codes = (v / scale[:, None]).view(-1, 16, v.shape[2]).transpose(1, 2).contiguous().to(E4M3)
    return {"codes": codes.flatten(), "scales": e.to(torch.uint8).flatten()}


def _unpacked(case, kept):
    rows, ld = _up(case["rows"], 32), _up(case["cols"], 16)
    codes = kept[:rows * ld].view(E4M3).float().view(-1, ld, 16).transpose(1, 2).reshape(-1, 32, ld)
    scale = (kept[rows * ld:].int() << 23).view(torch.float32).view(-1, 1, ld)
    return (codes * scale).view(-1, ld)[:case["rows"], :case["cols"]]


def _gradient(case, s):
    dw = s["dy"].float().t() @ _unpacked(case, s["kept"])
    return {"dw": dw.bfloat16() if case["out"] == "bf16" else dw}


# ------------------------------------------------------ the same in 64 bits

def _power(e):
    """2^e, exactly (whole e, 64 bits)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_grid(v):
    """The nearest e4m3 values (ties to even): 3 bits of fraction, exponents from -6 on."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = _power((e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = _inputs(case, seed)
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "int8":
        d = torch.mm(s["a"].double() * s["a_scale"].double()[:, None],
                     (s["b"].double() * s["b_scale"].double()[:, None]).t())
        return {"d": d + s["bias"].double() if case["bias"] else d}
    if case["op"] == "quantize":
        x = s["x"].double()
        top = x.abs().max(1).values
        v = x * TOP[case["out"]] / torch.where(top > 0, top, 1.0)[:, None]
        return {"q": torch.round(v).to(torch.int8) if case["out"] == "int8" else _e4m3_grid(v),
                "scale": top / TOP[case["out"]]}
    if case["op"] == "checkpoint":
        return _exact_checkpoint(case, s)
    parts = []
    weights = [torch.zeros(cols, dtype=torch.float64, device=DEVICE) for _ in range(2)]
    w = s["weight"].double()
    pw = s["post_weight"].double() if case["post"] else None
    for a in range(0, rows, 1024):
        t = {k: v[a:a + 1024].double() for k, v in s.items() if k not in ("weight", "post_weight")}
        gate = 1 / (1 + torch.exp(-t["z"])) if case["gate"] else 1.0
        got = {}
        if case["step"] == "forward":
            n = t["x"]
            if case["post"]:
                length = (n.pow(2).sum(1) / cols + EPS).pow(0.5)
                got["post_rstd"] = 1 / length
                n = n / length[:, None] * pw
            got["h"] = h = RESIDUAL * t["r"] + BRANCH * (gate * n)
            length = (h.pow(2).sum(1) / cols + EPS).pow(0.5)
            got["rstd"] = 1 / length
            y = h / length[:, None] * w
            if case["out"] == "e4m3":
                top = y.abs().max(1).values
                got["scale"] = top / 448
                y = _e4m3_grid(y / torch.where(top > 0, top, 1.0)[:, None] * 448)
            got["y"] = y
        else:
            n = t["h"] * t["rstd"][:, None]
            weights[0] += (t["dy"] * n).sum(0)
            inner = (t["dy"] * w * n).sum(1, keepdim=True) / cols
            d = (t["dy"] * w - inner * n) * t["rstd"][:, None] + t["dh"]
            got["dr"] = RESIDUAL * d
            d = BRANCH * d
            n = t["x"] * t["post_rstd"][:, None] if case["post"] else t["x"]
            if case["gate"]:
                got["dz"] = d * (n * pw if case["post"] else n) * (gate - gate * gate)
            d = d * gate
            if case["post"]:
                weights[1] += (d * n).sum(0)
                inner = (d * pw * n).sum(1, keepdim=True) / cols
                d = (d * pw - inner * n) * t["post_rstd"][:, None]
            got["dx"] = d
        parts.append(got)
    got = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["step"] == "backward":
        got["dweight"] = weights[0]
        if case["post"]:
            got["dpost_weight"] = weights[1]
    return got


def _exact_checkpoint(case, s):
    rows, cols = case["rows"], case["cols"]
    if case["step"] == "gradient":
        tokens, ld = _up(rows, 32), _up(cols, 16)
        x = s["kept"][:tokens * ld].view(E4M3).double().reshape(tokens // 16, ld, 16)
        x = x.permute(0, 2, 1).reshape(tokens, ld)
        power = s["kept"][tokens * ld:].reshape(tokens // 32, ld).int() - 127
        x = x * _power(power).repeat_interleave(32, 0)
        return {"dw": torch.mm(s["dy"].double().t().contiguous(), x[:rows, :cols].contiguous())}
    tokens, ld = _up(rows, 32), _up(cols, 16)
    x = torch.zeros((tokens, ld), dtype=torch.float64, device=DEVICE)
    x[:rows, :cols] = s["x"].double()
    x = x.reshape(tokens // 32, 32, ld)
    top = x.abs().max(1).values
    # The least power of two that brings the largest magnitude to 448 or below.
    power = torch.full(top.shape, -109, device=DEVICE)
    for p in range(-109, 120):
        power += top > 448 * 2.0 ** p
    power = power.clamp(max=119)
    codes = _e4m3_grid(x / _power(power)[:, None])
    codes = codes.reshape(tokens // 16, 16, ld).permute(0, 2, 1)
    return {"codes": codes.reshape(-1), "scales": (power + 127).to(torch.uint8).reshape(-1)}
