"""Timed cases of the calls on both sides of the vocabulary head: the root-mean-square norm that makes its hidden rows
(with the residual's addition, 8-bit rows for an 8-bit head, and its backward pass), the head's product in 8-bit
integers, and the cross entropy of the head's scores with its gradients, without the scores.

Each case runs in two forms: `own = False` computes the call from elementary torch operations in fp32, and
`own = True` makes the call a user makes of `top_sampling_apply_gb300`.  `exact` gives the same outputs from
the definitions in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a fine-tuning step's smallest micro-batch on a small head, where the launches count
        {"name": "xent_m16", "op": "xent", "M": 16, "V": 8192, "H": 1024, "bias": False, "cap": 0.0, "z": 0.0,
         "skip": 0.0},
        # instruction tuning: the prompt's tokens, a third of the rows, are not trained on
        {"name": "xent_m512", "op": "xent", "M": 512, "V": 32000, "H": 2048, "bias": False, "cap": 0.0, "z": 0.0,
         "skip": 0.33},
        # nothing round: a bias, capped scores, a penalty on the normaliser, odd rows and vocabulary
        {"name": "xent_odd", "op": "xent", "M": 1023, "V": 32001, "H": 2056, "bias": True, "cap": 30.0, "z": 1e-4,
         "skip": 0.05},
        # a pre-training micro-batch at the largest vocabulary
        {"name": "xent_m2048", "op": "xent", "M": 2048, "V": 128256, "H": 5120, "bias": False, "cap": 0.0, "z": 0.0,
         "skip": 0.0},
        # one decoded token before the head: the residual's addition, the norm and the row in 8 bits
        {"name": "norm_bf16_8bit_m1", "op": "norm", "M": 1, "H": 2048, "dtype": "bf16", "weight": "bf16",
         "residual": True, "bits": 8},
        # the last norm of a decode batch, rows in 8 bits
        {"name": "norm_bf16_8bit_m256", "op": "norm", "M": 256, "H": 5120, "dtype": "bf16", "weight": "bf16",
         "residual": True, "bits": 8},
        # a training step's forward pass over its whole batch
        {"name": "norm_bf16_m16384", "op": "norm", "M": 16384, "H": 5120, "dtype": "bf16", "weight": "bf16",
         "residual": True, "bits": 16},
        # its backward pass, with the gradient that comes along the residual
        {"name": "norm_back_bf16_m16384", "op": "norm_back", "M": 16384, "H": 5120, "dtype": "bf16",
         "weight": "bf16", "residual": True},
        # an odd width in fp32 with no residual
        {"name": "norm_back_f32_odd", "op": "norm_back", "M": 1001, "H": 2051, "dtype": "f32", "weight": "f32",
         "residual": False},
        # the scores of one decoded token, for `sample`
        {"name": "int8_m1", "op": "int8", "M": 1, "V": 32000, "H": 2048, "dtype": "bf16", "bias": False},
        # the scores of a decode batch at the largest vocabulary
        {"name": "int8_m64", "op": "int8", "M": 64, "V": 128256, "H": 5120, "dtype": "bf16", "bias": False},
        # the scores of every position of a batch of prompts, fp32 for their log-probabilities, a bias, ragged sizes
        {"name": "int8_m2047_f32", "op": "int8", "M": 2047, "V": 32001, "H": 4112, "dtype": "f32", "bias": True},
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["xent", "xent", "xent", "norm", "norm", "norm_back", "norm_back", "int8", "int8", "int8"])
    if op in ("norm", "norm_back"):
        H = _between(rng, 64, 16384)
        dtype = rng.choice(["f32", "f16", "bf16"])
        case = {"op": op, "M": _between(rng, 1, min(16384, 80_000_000 // H)), "H": H, "dtype": dtype,
                "weight": rng.choice([dtype, "f32"]), "residual": rng.random() < 0.6}
        if op == "norm":
            case["bits"] = rng.choice([8, 16])
        return case
    V = _between(rng, 1000, 128000)
    if op == "int8":
        H = 16 * _between(rng, 16, 512)
        return {"op": op, "M": _between(rng, 1, min(2048, 300_000_000_000 // (V * H))), "V": V, "H": H,
                "dtype": rng.choice(["f32", "f16", "bf16"]), "bias": rng.random() < 0.4}
    H = 8 * _between(rng, 16, 512)
    return {"op": op, "M": _between(rng, 1, min(4096, 500_000_000_000 // (V * H))), "V": V, "H": H,
            "bias": rng.random() < 0.3, "cap": rng.choice([0.0, 0.0, 30.0]), "z": rng.choice([0.0, 1e-4]),
            "skip": rng.choice([0.0, 0.1, 0.5])}


def _skipped(case):
    return int(case["M"] * case["skip"])


def work(case):
    op, M, H = case["op"], case["M"], case["H"]
    if op == "xent":
        V, n = case["V"], M - _skipped(case)
        # the weight and the rows that count, and the gradients of all; products for the scores and both gradients
        b = 2 * 2 * V * H + 2 * n * H + 2 * M * H + 16 * M + (8 * V if case["bias"] else 0)
        return {"bytes": b, "flops": 6 * n * V * H}
    if op == "norm":
        es, ws = (4 if case["dtype"] == "f32" else 2), (4 if case["weight"] == "f32" else 2)
        # the row, and with a residual that and their sum; the result, in 8 bits a byte and a scale a row
        b = M * H * es * (3 if case["residual"] else 1) + M * H * (1 if case["bits"] == 8 else es) + ws * H + 8 * M
        return {"bytes": b, "flops": 6 * M * H}
    if op == "norm_back":
        es, ws = (4 if case["dtype"] == "f32" else 2), (4 if case["weight"] == "f32" else 2)
        return {"bytes": M * H * es * (4 if case["residual"] else 3) + 2 * ws * H + 4 * M, "flops": 10 * M * H}
    V, es = case["V"], (4 if case["dtype"] == "f32" else 2)
    return {"bytes": V * H + M * H + M * V * es + 4 * M + 4 * V + (4 * V if case["bias"] else 0),
            "flops": 2 * M * V * H}


# ------------------------------------------------------------------ inputs
EPS = 1e-6


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _codes(n, H, g):
    """Rows of 8-bit codes as a normal row's are: a largest of 127 and a deviation of about 32."""
    q = torch.empty(n, H, dtype=torch.int8, device=DEV)
    q.copy_(torch.randn(n, H, generator=g, device=DEV).mul_(32.0).round_().clamp_(-127, 127))
    q[:, H // 2] = 127
    return q


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op, M, H = case["op"], case["M"], case["H"]
    if op in ("norm", "norm_back"):
        dt = DT[case["dtype"]]
        # a residual stream: some channels are many times the others
        size = torch.randn(H, generator=g, device=DEV).mul_(0.5).exp_()
        s["x"] = torch.randn(M, H, generator=g, device=DEV).mul_(size).to(dt)
        s["w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(DT[case["weight"]])
        s["r"] = None
        if case["residual"]:
            s["r"] = torch.randn(M, H, generator=g, device=DEV).mul_(size).mul_(2.0).to(dt)
        if op == "norm_back":
            # `r` is the gradient along the residual here
            s["dy"] = torch.randn(M, H, generator=g, device=DEV).mul_(0.01).to(dt)
            if s["r"] is not None:
                s["r"] = (s["r"].float() * 0.01).to(dt)
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(-1) + EPS).float()
        return s
    V = case["V"]
    s["b"] = torch.randn(V, generator=g, device=DEV) if case["bias"] else None
    if op == "int8":
        s["h"], s["weight"] = _codes(M, H, g), _codes(V, H, g)
        s["hs"] = (torch.rand(M, generator=g, device=DEV) + 0.5) / 32.0
        s["ws"] = (torch.rand(V, generator=g, device=DEV) + 0.5) * (3.0 / 32.0 / math.sqrt(H))
        return s
    s["h"] = torch.randn(M, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    s["weight"] = w.normal_(0.0, 3.0 / math.sqrt(H), generator=g)
    s["targets"] = torch.randint(0, V, (M,), generator=g, device=DEV)
    skip = torch.randperm(M, generator=g, device=DEV)[:_skipped(case)]
    s["targets"][skip] = -1
    return s


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    x = s["x"].float()
    out = {}
    if s["residual"]:
        # the norm is of the sum as the stream holds it
        out["residual"] = (x + s["r"].float()).to(s["x"].dtype)
        x = out["residual"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(-1) + EPS)
    y = x * rstd[:, None] * s["w"].float()
    out["rstd"] = rstd
    if s["bits"] == 8:
        scale = y.abs().amax(-1) / 127.0
        q = torch.round(y / scale[:, None])
        out["scale"] = scale
        out["y"] = (q * scale[:, None]).to(torch.bfloat16)
    else:
        out["y"] = y.to(s["x"].dtype)
    return out


def _plain_norm_back(s):
    x = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    f = dy * s["w"].float()
    dx = (f - x * (f * x).mean(-1, keepdim=True)) * s["rstd"][:, None]
    if s["residual"]:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * x).sum(0).to(s["w"].dtype)}


def _plain_int8(s):
    z = s["h"].float() @ s["weight"].float().t()
    z = z * s["hs"][:, None] * s["ws"]
    if s["b"] is not None:
        z = z + s["b"]
    return z.to(DT[s["dtype"]])


def _plain_xent(s):
    h, w, t = s["h"].float(), s["weight"].float(), s["targets"]
    live = t >= 0
    n = live.sum()
    row_w = torch.where(live, 1.0 / torch.clamp(n, min=1).float(), 0.0)
    z = h @ w.t()
    if s["b"] is not None:
        z = z + s["b"]
    slope = None
    if s["cap"] > 0:
        z = torch.tanh(z / s["cap"])
        slope = 1.0 - z * z
        z = z * s["cap"]
    top = z.amax(-1)
    lse = top + (z - top[:, None]).exp().sum(-1).log()
    at = t.clamp(min=0)[:, None]
    row = lse - z.gather(1, at)[:, 0] + s["z"] * lse * lse
    row = torch.where(live, row, 0.0)
    f = (z - lse[:, None]).exp() * (row_w * (1.0 + 2.0 * s["z"] * lse))[:, None]
    del z
    f.scatter_add_(1, at, -row_w[:, None])
    if slope is not None:
        f = f * slope
    out = {"loss": (row_w * row).sum(), "row": row, "lse": torch.where(live, lse, 0.0)}
    out["dh"] = (f @ w).to(torch.bfloat16)
    out["dw"] = (f.t() @ h).to(torch.bfloat16)
    if s["b"] is not None:
        out["db"] = f.sum(0)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if not own:
        return {"norm": _plain_norm, "norm_back": _plain_norm_back, "int8": _plain_int8, "xent": _plain_xent}[op](s)
    import top_sampling_apply_gb300 as tsa

    if op == "norm":
        r = tsa.rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, quantize=s["bits"] == 8)
        out = {"rstd": r.rstd}
        if s["residual"]:
            out["residual"] = r.residual
        if s["bits"] == 8:
            # the values that the codes stand for
            y = torch.empty(r.out.shape, dtype=torch.bfloat16, device=r.out.device)
            out["y"] = torch.mul(r.out, r.scale[:, None], out=y)
            out["scale"] = r.scale
        else:
            out["y"] = r.out
        return out
    if op == "norm_back":
        dx, dw = tsa.rms_norm_backward(s["dy"], s["x"], s["w"], s["rstd"], grad_residual=s["r"])
        return {"dx": dx, "dw": dw}
    if op == "int8":
        return tsa.lm_head_int8(s["h"], s["hs"], s["weight"], s["ws"], bias=s["b"], dtype=DT[s["dtype"]])
    r = tsa.lm_head_cross_entropy(s["h"], s["weight"], s["targets"], bias=s["b"], softcap=s["cap"], z_loss=s["z"])
    out = {"loss": r.loss, "row": r.row_loss, "lse": r.lse, "dh": r.grad_hidden, "dw": r.grad_weight}
    if s["b"] is not None:
        out["db"] = r.grad_bias
    return out


# ------------------------------------------------------------------ fp64
def _exact_norm(s):
    x = s["x"].double()
    out = {}
    if s["residual"]:
        out["residual"] = x + s["r"].double()
        x = out["residual"].to(s["x"].dtype).double()
    mean = torch.linalg.vector_norm(x, dim=-1) ** 2 / s["H"]
    out["rstd"] = (mean + EPS) ** -0.5
    y = torch.einsum("mh,m,h->mh", x, out["rstd"], s["w"].double())
    if s["bits"] == 16:
        out["y"] = y
        return out
    out["scale"] = torch.maximum(y.amax(-1), -y.amin(-1)) / 127
    out["y"] = torch.round(y / out["scale"][:, None]) * out["scale"][:, None]
    return out


def _exact_norm_back(s):
    # by differentiating the definition, with the stored reciprocal root put where it was used
    x = s["x"].double().requires_grad_(True)
    w = s["w"].double().requires_grad_(True)
    y = x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w
    dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
    return {"dx": dx + s["r"].double() if s["residual"] else dx, "dw": dw}


def _exact_int8(s):
    z = torch.einsum("mh,vh->mv", s["h"].double(), s["weight"].double())
    z = z * torch.outer(s["hs"].double(), s["ws"].double())
    return z if s["b"] is None else z + s["b"].double()


def _exact_xent(s):
    live = (s["targets"] >= 0).nonzero()[:, 0]
    t = s["targets"][live]
    h = s["h"].double().requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    leaves = [h, w]
    y = h[live] @ w.t()
    if s["b"] is not None:
        leaves.append(s["b"].double().requires_grad_(True))
        y = y + leaves[-1]
    if s["cap"] > 0:
        y = torch.tanh(y / s["cap"]) * s["cap"]
    lse = torch.logsumexp(y, -1)
    row = lse - y[torch.arange(len(t), device=DEV), t] + s["z"] * lse ** 2
    loss = row.mean() if len(t) else row.sum()
    grads = torch.autograd.grad(loss, leaves)
    out = {"loss": loss.detach(), "dh": grads[0], "dw": grads[1]}
    if s["b"] is not None:
        out["db"] = grads[2]
    for name, x in (("row", row), ("lse", lse)):
        out[name] = torch.zeros(s["M"], dtype=torch.float64, device=DEV)
        out[name][live] = x.detach()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_back": _exact_norm_back, "int8": _exact_int8, "xent": _exact_xent}[case["op"]](s)
