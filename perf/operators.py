"""Timed cases of the training-side calls that sit next to the sampler: the clipped policy loss and the
preference loss with their gradients on the logits, the AdamW step over many tensors, and the log-probability
of a token straight from the hidden rows.

Each case runs in two forms: `own = False` computes the call from elementary torch operations in fp32, and
`own = True` makes the call a user makes of `top_sampling_apply_gb300`.  `exact` gives the same outputs from
the definitions in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 256  # elements that share one exponent in the 8-bit states


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest update: a handful of tokens of a small vocabulary, where the launches count
        {"name": "policy_f32_b8", "op": "policy", "B": 8, "V": 8192, "dtype": "f32", "ref": False, "pad": 0.0,
         "mask": False, "rowT": False, "entropy": False, "grad": True},
        # one training step's tokens of rollouts in bf16, an eighth of them padding, KL to a reference policy
        {"name": "policy_bf16_b4096", "op": "policy", "B": 4096, "V": 128256, "dtype": "bf16", "ref": True,
         "pad": 0.125, "mask": False, "rowT": False, "entropy": False, "grad": True},
        # grammar-constrained rollouts: odd vocabulary (rows at every alignment), masks, temperatures, entropy bonus
        {"name": "policy_f16_masked", "op": "policy", "B": 1023, "V": 32001, "dtype": "f16", "ref": True,
         "pad": 0.05, "mask": True, "rowT": True, "entropy": True, "grad": True},
        # the loss of held-out rollouts, no gradient, with the entropies
        {"name": "policy_f32_eval", "op": "policy", "B": 512, "V": 128256, "dtype": "f32", "ref": True, "pad": 0.0,
         "mask": False, "rowT": False, "entropy": True, "grad": False},
        # a few short pairs of a small vocabulary (one-token answers among them)
        {"name": "preference_bf16_small", "op": "preference", "P": 4, "lo": 1, "hi": 24, "V": 8192, "dtype": "bf16",
         "ref": True, "pad": 0.0, "average": False},
        # a training step's pairs at the largest vocabulary, prompt tokens weighted 0
        {"name": "preference_bf16_large", "op": "preference", "P": 8, "lo": 64, "hi": 448, "V": 128256,
         "dtype": "bf16", "ref": True, "pad": 0.25, "average": False},
        # length-normalised and reference-free, odd vocabulary, f32 logits
        {"name": "preference_f32_average", "op": "preference", "P": 24, "lo": 5, "hi": 90, "V": 32003,
         "dtype": "f32", "ref": False, "pad": 0.1, "average": True},
        # many small tensors (biases, norms, small matrices): one call for all of them
        {"name": "adamw_f32_small_tensors", "op": "adamw", "tensors": 150, "total": 1_000_000, "bits": 32,
         "param": "f32", "grad": "f32"},
        # a model of fp32 weights with fp32 states
        {"name": "adamw_f32_100m", "op": "adamw", "tensors": 60, "total": 100_000_000, "bits": 32, "param": "f32",
         "grad": "f32"},
        # bf16 weights and gradients with 8-bit states, the form for the largest models; then the states' values
        # as a checkpoint writes them
        {"name": "adamw_bf16_8bit_256m", "op": "adamw", "tensors": 96, "total": 256_000_000, "bits": 8,
         "param": "bf16", "grad": "bf16"},
        # the log-probability of one decoded token
        {"name": "lm_head_m1", "op": "lm_head", "M": 1, "V": 32000, "H": 2048, "bias": False, "cap": 0.0,
         "mask": False},
        # the log-probabilities of a rollout batch under a reference model
        {"name": "lm_head_m2048", "op": "lm_head", "M": 2048, "V": 128256, "H": 5120, "bias": True, "cap": 30.0,
         "mask": False},
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "policy", "preference", "preference", "adamw", "adamw", "lm_head", "lm_head"])
    if op == "policy":
        dtype = rng.choice(["f32", "f16", "bf16"])
        V = _between(rng, 2000, 160000)
        most = 500_000_000 // (V * (2 if dtype == "f32" else 1))
        return {"op": op, "B": _between(rng, 1, min(4096, most)), "V": V, "dtype": dtype,
                "ref": rng.random() < 0.6, "pad": rng.choice([0.0, 0.1, 0.3]), "mask": rng.random() < 0.4,
                "rowT": rng.random() < 0.4, "entropy": rng.random() < 0.5, "grad": rng.random() < 0.8}
    if op == "preference":
        dtype = rng.choice(["f32", "f16", "bf16"])
        V = _between(rng, 2000, 130000)
        lo = _between(rng, 1, 40)
        hi = lo + _between(rng, 1, 200)
        most = max(1, 400_000_000 // (V * (2 if dtype == "f32" else 1)) // (2 * hi))
        avg = rng.random() < 0.4
        return {"op": op, "P": _between(rng, 1, min(64, most)), "lo": lo, "hi": hi, "V": V, "dtype": dtype,
                "ref": not avg, "pad": rng.choice([0.0, 0.2]), "average": avg}
    if op == "adamw":
        bits = rng.choice([8, 32])
        total = _between(rng, 300_000, 100_000_000)
        return {"op": op, "tensors": _between(rng, 1, 400), "total": total, "bits": bits,
                "param": rng.choice(["f32", "bf16"]), "grad": rng.choice(["f32", "bf16"])}
    V = _between(rng, 8000, 130000)
    H = 8 * _between(rng, 32, 512)
    return {"op": op, "M": _between(rng, 1, 2048), "V": V, "H": H, "bias": rng.random() < 0.5,
            "cap": rng.choice([0.0, 30.0]), "mask": rng.random() < 0.4}


def _lengths(case):
    """Tokens of each sequence: the P chosen ones, then the P rejected ones."""
    r = random.Random("%d-%d-%d" % (case["P"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(2 * case["P"])]


def _sizes(case):
    """Elements of each tensor: spread over four decades, every other one odd."""
    n, total = case["tensors"], case["total"]
    r = random.Random("%d-%d" % (n, total))
    w = [math.exp(r.uniform(0.0, 9.0)) for _ in range(n)]
    k = total / sum(w)
    out = []
    for i, x in enumerate(w):
        size = max(1, int(x * k))
        out.append(size | 1 if i % 2 else max(64, size // 64 * 64))
    return out


def _skipped(case, n):
    return int(n * case["pad"])


def work(case):
    op = case["op"]
    if op == "policy":
        es, B, V = (4 if case["dtype"] == "f32" else 2), case["B"], case["V"]
        read = B - _skipped(case, B)
        n = read * V * es + 40 * B
        if case["mask"]:
            n += read * ((V + 31) // 32) * 4
        if case["grad"]:
            n += B * V * es
        return {"bytes": n, "flops": read * V * (10 if case["grad"] else 5)}
    if op == "preference":
        es, V, N = (4 if case["dtype"] == "f32" else 2), case["V"], sum(_lengths(case))
        read = N - _skipped(case, N)
        return {"bytes": read * V * es + N * V * es + 24 * N, "flops": read * V * 10}
    if op == "adamw":
        n = sum(_sizes(case))
        ps, gs = (4 if case["param"] == "f32" else 2), (4 if case["grad"] == "f32" else 2)
        # 8 bits: codes in and out, and the values of both states written in bf16
        state = 16 if case["bits"] == 32 else 4 + 4
        return {"bytes": n * (2 * ps + gs + state), "flops": n * 15}
    M, V, H = case["M"], case["V"], case["H"]
    n = 2 * V * H + 2 * M * H + 12 * M + (4 * V if case["bias"] else 0) + (M * ((V + 31) // 32) * 4 if case["mask"] else 0)
    return {"bytes": n, "flops": 2 * M * V * H}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _pack(allowed):
    """bool [B, V] -> int32 [B, ceil(V / 32)], token i at bit i % 32 of word i // 32."""
    B, V = allowed.shape
    W = (V + 31) // 32
    bits = torch.zeros(B, W * 32, dtype=torch.int64, device=allowed.device)
    bits[:, :V] = allowed
    word = (bits.view(B, W, 32) << torch.arange(32, device=allowed.device)).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def _unpack(mask, V):
    bits = (mask.unsqueeze(-1) >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1
    return bits.reshape(mask.shape[0], -1)[:, :V] != 0


def _logits(N, V, dtype, g):
    """Normal logits over a head that falls with the logarithm of the token's rank, as language models give."""
    rank = torch.randperm(V, generator=g, device=DEV).float().add_(1.0)
    x = torch.randn(N, V, generator=g, device=DEV).mul_(2.0).sub_(rank.log_().mul_(1.1))
    return x.to(dtype)


def _token_and_logprob(x, T, allowed, g):
    """A token drawn from each row and its log-probability."""
    y = x.float() / T
    if allowed is not None:
        y = y.masked_fill(~allowed, -math.inf)
    e = torch.empty_like(y).exponential_(generator=g)
    tok = (y - e.log_()).argmax(-1)
    return tok, y.gather(1, tok[:, None])[:, 0] - torch.logsumexp(y, -1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "policy":
        B, V = case["B"], case["V"]
        s = dict(case)
        x = _logits(B, V, DT[case["dtype"]], g)
        T = torch.rand(B, 1, generator=g, device=DEV) * 0.9 + 0.6 if case["rowT"] else torch.ones(B, 1, device=DEV)
        allowed = torch.rand(B, V, generator=g, device=DEV) < 0.5 if case["mask"] else None
        tok, lp = _token_and_logprob(x, T, allowed, g)
        s["old"] = lp + 0.15 * torch.randn(B, generator=g, device=DEV)
        s["adv"] = torch.randn(B, generator=g, device=DEV) + 0.4
        s["ref_lp"] = lp + 0.3 * torch.randn(B, generator=g, device=DEV) if case["ref"] else None
        w = torch.full((B,), 1.0 / B, device=DEV)
        skip = torch.randperm(B, generator=g, device=DEV)[:_skipped(case, B)]
        w[skip] = 0.0
        # what padding rows hold is nobody's business: leave one of them full of NaN
        x[skip[:1]] = math.nan
        if case["mask"] and B >= 8:
            # a row that allows nothing (token -1, as `sample` gives) and a row whose token its mask excludes
            allowed[B - 1] = False
            tok[B - 1] = -1
            allowed[B - 2, tok[B - 2]] = False
        s.update(logits=x, tokens=tok, w=w, T=T[:, 0].contiguous() if case["rowT"] else 1.0,
                 bits=_pack(allowed) if case["mask"] else None, kl=0.04 if case["ref"] else 0.0,
                 ent=0.01 if case["entropy"] else 0.0)
        return s
    if op == "preference":
        n = _lengths(case)
        N, V = sum(n), case["V"]
        s = dict(case)
        x = _logits(N, V, DT[case["dtype"]], g)
        tok, lp = _token_and_logprob(x, torch.ones(N, 1, device=DEV), None, g)
        start = [0]
        for k in n:
            start.append(start[-1] + k)
        w = torch.ones(N, device=DEV)
        w[torch.randperm(N, generator=g, device=DEV)[:_skipped(case, N)]] = 0.0
        s.update(logits=x, tokens=tok, w=w, start=torch.tensor(start, dtype=torch.int64, device=DEV),
                 ref_lp=lp + 0.2 * torch.randn(N, generator=g, device=DEV) if case["ref"] else None,
                 beta=2.0 if case["average"] else 0.1, margin=0.5 if case["average"] else 0.0,
                 smooth=0.0 if case["average"] else 0.1)
        return s
    if op == "adamw":
        sizes = _sizes(case)
        start = [0]
        for k in sizes:
            start.append(start[-1] + (k + BLOCK - 1) // BLOCK * BLOCK)
        total = start[-1]
        live = torch.zeros(total, dtype=torch.bool, device=DEV)
        edges = torch.zeros(total + 1, dtype=torch.int32, device=DEV)
        a = torch.tensor(start[:-1], device=DEV)
        edges[a] += 1
        edges[a + torch.tensor(sizes, device=DEV)] -= 1
        live = edges.cumsum(0)[:total] > 0
        # gradients of a few thousandths whose size differs from tensor part to tensor part
        size = torch.randn(total // BLOCK, generator=g, device=DEV).exp_().repeat_interleave(BLOCK)
        grad = torch.randn(total, generator=g, device=DEV).mul_(size).mul_(2e-3).mul_(live)
        p = torch.randn(total, generator=g, device=DEV).mul_(0.05).mul_(live)
        m = torch.randn(total, generator=g, device=DEV).mul_(size).mul_(4e-4).mul_(live)
        v = (torch.randn(total, generator=g, device=DEV).abs_() + 0.1).mul_(size).mul_(2e-3).square_().mul_(live)
        s = dict(case, sizes=sizes, start=start, t=100, p=p.to(DT[case["param"]]), g=grad.to(DT[case["grad"]]),
                 scale=torch.full((1,), 0.5, device=DEV), seed=seed & 0xFFFF, me=None, ve=None)
        if case["bits"] == 32:
            s.update(m=m, v=v)
        else:
            s["m"], s["me"] = _to8(m, False, None)
            s["v"], s["ve"] = _to8(v, True, torch.full_like(v, 0x8000, dtype=torch.int32))
            s["out_m"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
            s["out_v"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV)
        if own:
            import top_sampling_apply_gb300 as tsa

            def cut(t, blocks=False):
                if t is None:
                    return None
                if blocks:
                    return [t[b // BLOCK:b // BLOCK + (k + BLOCK - 1) // BLOCK] for b, k in zip(start, sizes)]
                return [t[b:b + k] for b, k in zip(start, sizes)]

            s["plan"] = tsa.adamw_plan(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), cut(s["me"], True),
                                       cut(s["ve"], True))
            if case["bits"] == 8:
                s["outs"] = (cut(s["out_m"]), cut(s["out_v"]))
        return s
    M, V, H = case["M"], case["V"], case["H"]
    s = dict(case)
    s["h"] = torch.randn(M, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    s["weight"] = w.normal_(0.0, 3.0 / math.sqrt(H), generator=g)
    s["b"] = torch.randn(V, generator=g, device=DEV) if case["bias"] else None
    s["tokens"] = torch.randint(0, V, (M,), generator=g, device=DEV)
    s["bits"] = None
    if case["mask"]:
        allowed = torch.rand(M, V, generator=g, device=DEV) < 0.5
        allowed[torch.arange(M, device=DEV), s["tokens"]] = True
        s["bits"] = _pack(allowed)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_rows(x, T, allowed):
    """ln p of every entry of the allowed, temperature-scaled rows (-inf where not allowed)."""
    x = x.float() / T
    x = torch.where(torch.isnan(x), -math.inf, x)
    if allowed is not None:
        x = torch.where(allowed, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x - top
    return x - x.exp().sum(-1, keepdim=True).log()


def _plain_policy(s):
    x, V = s["logits"], s["V"]
    T = s["T"][:, None] if s["rowT"] else 1.0
    lp = _plain_rows(x, T, _unpack(s["bits"], V) if s["mask"] else None)
    tok = s["tokens"]
    named = (s["w"] != 0) & (tok >= 0) & (tok < V)
    at = tok.clamp(0, V - 1)[:, None]
    l = lp.gather(1, at)[:, 0]
    live = named & (l > -math.inf)
    d = torch.where(live, l - s["old"], 0.0)
    r = d.exp()
    A = torch.where(live, s["adv"], 0.0)
    s1, s2 = r * A, r.clamp(0.8, 1.2) * A
    row = -torch.minimum(s1, s2)
    c = torch.where(s1 <= s2, -s1, torch.zeros_like(s1))
    if s["ref"]:
        u = torch.where(live, s["ref_lp"] - l, 0.0)
        row = row + s["kl"] * (u.exp() - u - 1.0)
        c = c + s["kl"] * (1.0 - u.exp())
    H = None
    p = lp.exp()
    if s["entropy"]:
        H = -torch.where(p > 0, p * lp, 0.0).sum(-1)
        H = torch.where(live, H, 0.0)
        row = row - s["ent"] * H
    row = torch.where(live, row, 0.0)
    w = torch.where(live, s["w"], 0.0)
    out = {"loss": (w * row).sum(), "row": row, "logprob": torch.where(named, l, 0.0)}
    if s["entropy"]:
        out["entropy"] = H
    if s["grad"]:
        f = (-c)[:, None] * p
        if s["entropy"]:
            f = f + torch.where(p > 0, s["ent"] * p * (lp + H[:, None]), 0.0)
        f.scatter_add_(1, at, c[:, None])
        f = f * (w[:, None] / T)
        out["grad"] = torch.where(live[:, None], f, 0.0).to(x.dtype)
    return out


def _plain_preference(s):
    x, V, P = s["logits"], s["V"], s["P"]
    lp = _plain_rows(x, 1.0, None)
    at = s["tokens"][:, None]
    l = lp.gather(1, at)[:, 0]
    w, start = s["w"], s["start"]
    live = w != 0
    i = torch.arange(x.shape[0], device=x.device)
    member = ((i >= start[:-1, None]) & (i < start[1:, None])).float() * w
    gain = l - s["ref_lp"] if s["ref"] else l
    gain = torch.where(live, gain, 0.0)
    R = (member * gain).sum(-1)
    if s["average"]:
        n = member.sum(-1)
        inv = torch.where(n > 0, 1.0 / n, 0.0)
        R = R * inv
    h = s["beta"] * (R[:P] - R[P:]) - s["margin"]
    e = s["smooth"]
    soft = lambda z: torch.maximum(z, torch.zeros_like(z)) + torch.log1p(torch.exp(-z.abs()))  # noqa: E731
    pair = (1.0 - e) * soft(-h) + e * soft(h)
    dh = -(1.0 - e) / (1.0 + h.exp()) + e / (1.0 + (-h).exp())
    dR = torch.cat([dh, -dh]) * (s["beta"] / P)
    if s["average"]:
        dR = dR * inv
    c = (member * dR[:, None]).sum(0)
    f = -c[:, None] * lp.exp()
    f.scatter_add_(1, at, c[:, None])
    return {"loss": pair.sum() / P, "pair": pair, "reward": s["beta"] * R, "logprob": torch.where(live, l, 0.0),
            "grad": torch.where(live[:, None], f, 0.0).to(x.dtype)}


def _philox(q, row, seed, offset):
    """The four 32-bit words of Philox4x32-10 for counters (q, row, offset, 0) under key (seed, 0), as int64."""
    low = 0xFFFFFFFF

    def mul(a, c):
        hi = (a * (c >> 16) + ((a * (c & 0xFFFF)) >> 16)) >> 16
        return hi & low, (a * c) & low

    c = [q & low, row, torch.full_like(q, offset), torch.zeros_like(q)]
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        ah, al = mul(0xD2511F53, c[0])
        dh, dl = mul(0xCD9E8D57, c[2])
        c = [dh ^ c[1] ^ k0, dl, ah ^ c[3] ^ k1, al]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _words(s):
    """The random word of every element of the flat buffers, as int32-ranged int64."""
    start = torch.tensor(s["start"], device=DEV)
    quads = (start[1:] - start[:-1]) // 4
    row = torch.repeat_interleave(torch.arange(len(s["sizes"]), device=DEV), quads)
    q = torch.arange(row.numel(), device=DEV) - (start[:-1] // 4)[row]
    return torch.stack(_philox(q, row, s["seed"], s["t"]), -1).reshape(-1)


def _to8(x, unsigned, r):
    """Codes and block exponents.  A block's base is (largest biased exponent) - 30 (unsigned, 5 exponent bits) or
    - 14 (signed, 4), at least 0; a code is the float's exponent and first three mantissa bits above the base.
    Unsigned codes are rounded by the 16 random bits r and never fall to 0 for a value above 0; signed ones to
    the nearest, ties to even."""
    bits = x.abs().view(torch.int32)
    top = bits.view(-1, BLOCK).amax(-1) >> 23
    base = (top - (30 if unsigned else 14)).clamp_min(0)
    b8 = (base * 8).repeat_interleave(BLOCK)
    if unsigned:
        code = ((bits + (r << 4)) >> 20) - b8
        code = torch.where(bits > 0, code.clamp(1, 255), 0)
    else:
        code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - b8
        code = code.clamp(0, 127) | torch.where(x < 0, 128, 0)
    return code.to(torch.uint8), base.to(torch.uint8)


def _from8(code, base, unsigned):
    c = code.to(torch.int32)
    mag = c if unsigned else c & 127
    b8 = (base.to(torch.int32) * 8).repeat_interleave(BLOCK)
    x = torch.where(mag > 0, (mag + b8) << 20, 0).view(torch.float32)
    return x if unsigned else torch.where(c > 127, -x, x)


LR, B1, B2, EPS, WD = 1e-3, 0.9, 0.999, 1e-8, 0.1


def _plain_adamw(s):
    wide = s["bits"] == 32
    word = _words(s) if not wide or s["param"] == "bf16" else None
    g = s["g"].float() * s["scale"]
    m, v = (s["m"], s["v"]) if wide else (_from8(s["m"], s["me"], False), _from8(s["v"], s["ve"], True))
    m = B1 * m + (1.0 - B1) * g
    v = B2 * v + (1.0 - B2) * (g * g)
    c1, c2 = 1.0 - B1 ** s["t"], 1.0 - B2 ** s["t"]
    p = s["p"].float() * (1.0 - LR * WD)
    p = p - (LR / c1) * (m / (v.sqrt() * (1.0 / math.sqrt(c2)) + EPS))
    if s["param"] == "bf16":
        bits = p.view(torch.int32)
        p = ((bits + (word >> 16).to(torch.int32)) & -65536).view(torch.float32)
    s["p"].copy_(p)
    s["t"] += 1
    if wide:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    for name, x, unsigned in (("m", m, False), ("v", v, True)):
        code, base = _to8(x, unsigned, (word & 0xFFFF).to(torch.int32))
        s[name].copy_(code)
        s[name + "e"].copy_(base)
    return {"p": s["p"], "m": _from8(s["m"], s["me"], False).to(torch.bfloat16),
            "v": _from8(s["v"], s["ve"], True).to(torch.bfloat16)}


def _plain_lm_head(s):
    z = s["h"].float() @ s["weight"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    if s["cap"] > 0:
        z = s["cap"] * torch.tanh(z / s["cap"])
    lp = _plain_rows(z, 1.0, _unpack(s["bits"], s["V"]) if s["mask"] else None)
    return lp.gather(1, s["tokens"][:, None])[:, 0]


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if not own:
        return {"policy": _plain_policy, "preference": _plain_preference, "adamw": _plain_adamw,
                "lm_head": _plain_lm_head}[op](s)
    import top_sampling_apply_gb300 as tsa

    if op == "policy":
        r = tsa.policy_loss(s["logits"], s["tokens"], s["old"], s["adv"], ref_logprob=s["ref_lp"], weight=s["w"],
                            clip_low=0.2, clip_high=0.2, kl_coef=s["kl"], entropy_coef=s["ent"], temperature=s["T"],
                            bitmask=s["bits"], return_entropy=s["entropy"], grad=s["grad"])
        out = {"loss": r.loss, "row": r.row_loss, "logprob": r.logprob}
        if s["entropy"]:
            out["entropy"] = r.entropy
        if s["grad"]:
            out["grad"] = r.grad
        return out
    if op == "preference":
        r = tsa.preference_loss(s["logits"], s["tokens"], s["start"], weight=s["w"], ref_logprob=s["ref_lp"],
                                beta=s["beta"], label_smoothing=s["smooth"], margin=s["margin"],
                                average=s["average"])
        return {"loss": r.loss, "pair": r.pair_loss, "reward": r.reward, "logprob": r.logprob, "grad": r.grad}
    if op == "adamw":
        tsa.adamw_step(s["plan"], s["t"], LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, grad_scale=s["scale"],
                       seed=s["seed"], offset=s["t"])
        s["t"] += 1
        if s["bits"] == 32:
            return {"p": s["p"], "m": s["m"], "v": s["v"]}
        tsa.adamw_state_values(s["plan"], *s["outs"])
        return {"p": s["p"], "m": s["out_m"], "v": s["out_v"]}
    return tsa.lm_head_logprob(s["h"], s["weight"], s["tokens"], bias=s["b"], softcap=s["cap"], bitmask=s["bits"])


# ------------------------------------------------------------------ fp64
def _exact_rows(x, T, allowed, tokens):
    x = x.double().div(T) if torch.is_tensor(T) else x.double() / T
    if allowed is not None:
        x = x.masked_fill(~allowed, -math.inf)
    return x


def _exact_policy(s):
    x, V, B = s["logits"], s["V"], s["B"]
    allowed = _unpack(s["bits"], V) if s["mask"] else None
    tok = s["tokens"]
    named = ((s["w"] != 0) & (tok >= 0) & (tok < V)).nonzero()[:, 0]
    z = torch.zeros(B, dtype=torch.float64, device=DEV)
    out = {"row": z.clone(), "logprob": z.clone()}
    ok = torch.ones(len(named), dtype=torch.bool, device=DEV)
    if allowed is not None:
        ok = allowed[named, tok[named]]
        out["logprob"][named[~ok]] = -math.inf
    rows = named[ok]
    t = tok[rows]
    leaf = x[rows].double().requires_grad_(s["grad"])
    y = leaf / s["T"][rows].double()[:, None] if s["rowT"] else leaf * 1.0
    if allowed is not None:
        y = y.masked_fill(~allowed[rows], -math.inf)
    lp = torch.log_softmax(y, -1)
    l = lp[torch.arange(len(rows), device=DEV), t]
    out["logprob"][rows] = l.detach()
    ratio = torch.exp(l - s["old"][rows].double())
    A = s["adv"][rows].double()
    row = -torch.minimum(ratio * A, ratio.clamp(0.8, 1.2) * A)
    if s["ref"]:
        u = s["ref_lp"][rows].double() - l
        row = row + s["kl"] * (torch.exp(u) - 1.0 - u)
    if s["entropy"]:
        H = torch.special.entr(torch.softmax(y, -1)).sum(-1)
        row = row - s["ent"] * H
        out["entropy"] = z.clone()
        out["entropy"][rows] = H.detach()
    out["row"][rows] = row.detach()
    loss = (s["w"][rows].double() * row).sum()
    out["loss"] = loss.detach()
    if s["grad"]:
        if s["entropy"]:
            # the entropy's own gradient, written out: d H / d y = -p (ln p + H)
            loss = loss + (s["w"][rows].double() * s["ent"] * H).sum()
        (grad,) = torch.autograd.grad(loss, leaf)
        if s["entropy"]:
            p = torch.softmax(y.detach(), -1)
            k = (s["w"][rows].double() * s["ent"])[:, None]
            k = k / s["T"][rows].double()[:, None] if s["rowT"] else k
            grad = grad + k * (p * H.detach()[:, None] - torch.special.entr(p))
        full = torch.zeros(B, V, dtype=torch.float64, device=DEV)
        full[rows] = grad
        out["grad"] = full
    return out


def _exact_preference(s):
    x, P, start = s["logits"], s["P"], s["start"].tolist()
    leaf = x.double().requires_grad_(True)
    lp = torch.log_softmax(leaf, -1)[torch.arange(x.shape[0], device=DEV), s["tokens"]]
    w = s["w"].double()
    gain = lp - s["ref_lp"].double() if s["ref"] else lp
    R = []
    for a, b in zip(start[:-1], start[1:]):
        r = (gain[a:b] * w[a:b]).sum()
        n = w[a:b].sum()
        R.append(r / n if s["average"] and float(n) > 0 else r)
    R = torch.stack(R)
    h = s["beta"] * (R[:P] - R[P:]) - s["margin"]
    ls = torch.nn.functional.logsigmoid
    pair = -(1.0 - s["smooth"]) * ls(h) - s["smooth"] * ls(-h)
    loss = pair.mean()
    (grad,) = torch.autograd.grad(loss, leaf)
    return {"loss": loss.detach(), "pair": pair.detach(), "reward": s["beta"] * R.detach(),
            "logprob": torch.where(w != 0, lp.detach(), 0.0), "grad": grad}


def _exact_8(x, unsigned, r):
    """What an 8-bit state stands for after a step, by its definition: the value on a grid of eight steps an
    octave, rounded by r (unsigned) or to the nearest, ties to even."""
    mag = x.abs()
    _, e = torch.frexp(mag)  # mag in [2^(e-1), 2^e)
    top = e.view(-1, BLOCK).masked_fill(mag.view(-1, BLOCK) == 0, -10000).amax(-1).repeat_interleave(BLOCK)
    step = torch.ldexp(torch.ones_like(mag), e - 4)
    q = mag / step
    q = torch.floor(q + r.double() / 65536.0) if unsigned else torch.round(q)
    y = q * step
    low = torch.ldexp(torch.ones_like(mag), top - (31 if unsigned else 15))  # the code-0 value of the block's base
    least = low * 1.125
    y = torch.where(y < least, least if unsigned else 0.0, y)
    return torch.where(mag == 0, 0.0, torch.sign(x) * y)


def _exact_adamw(s):
    word = _words(s)
    g = s["g"].double() * s["scale"].double()
    wide = s["bits"] == 32
    m, v = (s["m"], s["v"]) if wide else (_from8(s["m"], s["me"], False), _from8(s["v"], s["ve"], True))
    m = B1 * m.double() + (1 - B1) * g
    v = B2 * v.double() + (1 - B2) * g ** 2
    mh, vh = m / (1 - B1 ** s["t"]), v / (1 - B2 ** s["t"])
    p = s["p"].double()
    p = p - LR * WD * p - LR * mh / (vh.sqrt() + EPS)
    if s["param"] == "bf16":
        _, e = torch.frexp(p.abs())
        step = torch.ldexp(torch.ones_like(p), e - 8)
        p = torch.where(p == 0, 0.0, torch.sign(p) * torch.floor(p.abs() / step + (word >> 16).double() / 65536.0) * step)
    if wide:
        return {"p": p, "m": m, "v": v}
    r = word & 0xFFFF
    return {"p": p, "m": _exact_8(m, False, r), "v": _exact_8(v, True, r)}


def _exact_lm_head(s):
    z = s["h"].double() @ s["weight"].double().t()
    if s["b"] is not None:
        z += s["b"].double()
    if s["cap"] > 0:
        z = torch.tanh(z / s["cap"]) * s["cap"]
    if s["mask"]:
        z = z.masked_fill(~_unpack(s["bits"], s["V"]), -math.inf)
    return z[torch.arange(s["M"], device=DEV), s["tokens"]] - torch.logsumexp(z, -1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"policy": _exact_policy, "preference": _exact_preference, "adamw": _exact_adamw,
            "lm_head": _exact_lm_head}[case["op"]](s)
