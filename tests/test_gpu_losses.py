"""The policy and preference losses on the GPU against their float64 definitions.

Tolerances, for u = 2^-24 (the fp32 unit roundoff):
  - an exponential's relative error: its argument (l - m) c2 carries two roundings, c2 one more, so
    3 u |ln e_j|; ex2.approx adds 2^-22.  Terms that matter to Z have |ln e_j| < 30.
  - Z is a sum of V such terms; its longest chain of additions in one thread is V / 128 (128 threads
    at least take part), then 12 merging steps of three roundings each.
  So ln Z, and a log-probability, is off by at most EPS(V) = (90 + 4 + V / 128 + 36) u, plus 3 u |lp| for
  the final subtraction's terms.
  - a row's loss moves with lp by its slope c, whose terms are each rounded a few times.
  - a gradient element is a p_j (+ b p_j (ln p_j + H)) with p_j's relative error EPS(V) + 3 u |ln p_j|,
    and a moves with lp by at most |A| r + kl e^u; then one rounding to the output type.
"""
import numpy as np
import pytest
import torch

from oracle import losses

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
OUT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-38}


@pytest.fixture(scope="module")
def tsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import top_sampling_apply_gb300 as lib

    lib.load_library()
    return lib


def eps(V):
    return (130 + V / 128) * U


def pack(allowed):
    B, V = allowed.shape
    W = (V + 31) // 32
    full = np.ones((B, W * 32), bool)  # bits past V set: they are ignored
    full[:, :V] = allowed
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)


def rows(rng, B, V, dtype, scale=3.0):
    x = torch.from_numpy((scale * rng.standard_normal((B, V))).astype(np.float32)).to(dtype)
    return x, x.double().numpy()


def f32(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(DEV)


def check(name, got, want, tol):
    got = got.double().cpu().numpy() if torch.is_tensor(got) else np.float64(got)
    want = np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), name
    bad = np.abs(got - want)[fin] > np.broadcast_to(tol, want.shape)[fin]
    assert not bad.any(), "%s: %d off, worst %g" % (name, bad.sum(), np.abs(got - want)[fin].max())


def check_policy(r, ref, V, dtype, adv, old, refl, w, T, kl, ent, grad=True):
    B = len(ref["row_loss"])
    lp = np.where(np.isfinite(ref["logprob"]), ref["logprob"], 0.0)
    tl = eps(V) + 3 * U * np.abs(lp)
    check("logprob", r.logprob, ref["logprob"], tl)
    ratio = np.exp(lp - old)
    ku = kl * (np.exp(refl - lp) + np.abs(refl - lp)) if refl is not None else 0.0
    mag = np.abs(adv) * ratio * (1 + np.abs(lp - old)) + ku  # what the slope and the loss are made of
    th = 4 * eps(V) * (1 + ref["entropy"])
    tr = mag * (2 * tl + 8 * U) + ent * th + 4 * U * np.abs(ref["row_loss"])
    check("row_loss", r.row_loss, ref["row_loss"], tr)
    check("loss", r.loss.reshape(1), [ref["loss"]], (np.abs(w) * tr).sum() + 2 * U * abs(ref["loss"]) + 1e-30)
    if r.entropy is not None:
        check("entropy", r.entropy, ref["entropy"], th)
    if not grad:
        assert r.grad is None
        return
    s = (np.abs(w) / np.where(np.asarray(T) > 0, T, 1.0))[:, None]
    g = np.abs(ref["grad"])
    # every part of an element is at most s (mag + ent (ln V + 1)) p_j; p_j <= 1, and small p_j have small parts
    top = s * (mag * 2 + ent * (1 + ref["entropy"]))[:, None]
    tg = g * (2 * OUT[dtype] + 4 * eps(V)) + top * 4 * (eps(V) + tl[:, None]) * np.minimum(1.0, ref["p"] + ref["hot"])
    check("grad", r.grad, ref["grad"], tg + TINY[dtype])
    assert np.all(r.grad.cpu().double().numpy()[ref["p"] + ref["hot"] == 0] == 0)  # masked entries exactly


def policy_case(rng, B, V, dtype, mask, rowT, kl, ent, scale=3.0):
    x, xd = rows(rng, B, V, dtype, scale)
    T = (0.5 + rng.random(B)).astype(np.float32) if rowT else np.float32(1.0)
    allowed = rng.random((B, V)) < 0.6 if mask else None
    tok = np.empty(B, np.int64)
    for b in range(B):
        y = xd[b] if allowed is None else np.where(allowed[b], xd[b], -np.inf)
        tok[b] = np.argmax(y + rng.gumbel(size=V)) if np.isfinite(y).any() else -1
    adv = rng.standard_normal(B).astype(np.float32)
    w = (rng.random(B) + 0.1).astype(np.float32)
    lp = losses.policy_loss(xd, tok, np.zeros(B), adv, T=T, allowed=allowed)["logprob"]
    old = (lp + 0.2 * rng.standard_normal(B)).astype(np.float32)
    refl = (lp + 0.4 * rng.standard_normal(B)).astype(np.float32) if kl else None
    return dict(x=x, xd=xd, tok=tok, adv=adv, w=w, old=old, refl=refl, T=T, allowed=allowed, kl=kl, ent=ent)


def reference(c, **kw):
    a = dict(weight=c["w"], kl=np.float32(c["kl"]), ent=np.float32(c["ent"]), T=c["T"], allowed=c["allowed"],
             clip_low=np.float64(np.float32(1) - np.float32(0.2)) * -1 + 1,
             clip_high=np.float64(np.float32(1) + np.float32(0.3)) - 1)
    ref = losses.policy_loss(c["xd"], c["tok"], c["old"], c["adv"], c["refl"], **{**a, **kw})
    B, V = c["xd"].shape
    T = np.broadcast_to(np.where(np.asarray(c["T"]) > 0, c["T"], 1.0), (B,))
    y = np.where(np.isnan(c["xd"]), -np.inf, c["xd"]) / T[:, None]
    if c["allowed"] is not None:
        y = np.where(c["allowed"], y, -np.inf)
    with np.errstate(invalid="ignore"):
        p = np.exp(y - y.max(1, keepdims=True))
    p = np.where(np.isfinite(p), p, 0.0)
    ref["p"] = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    ref["hot"] = np.zeros((B, V))
    ok = (c["tok"] >= 0) & (c["tok"] < V)
    ref["hot"][np.arange(B)[ok], c["tok"][ok]] = 1.0
    return ref


def call(tsa, c, x=None, **kw):
    T = torch.from_numpy(c["T"]).to(DEV) if np.ndim(c["T"]) else float(c["T"])
    a = dict(ref_logprob=None if c["refl"] is None else f32(c["refl"]), weight=f32(c["w"]), clip_low=0.2,
             clip_high=0.3, kl_coef=c["kl"], entropy_coef=c["ent"], temperature=T,
             bitmask=None if c["allowed"] is None else pack(c["allowed"]), return_entropy=c["ent"] != 0)
    x = c["x"].to(DEV) if x is None else x
    return tsa.policy_loss(x, torch.from_numpy(c["tok"]).to(DEV), f32(c["old"]), f32(c["adv"]), **{**a, **kw})


def verify(c, r, **kw):
    ref = reference(c)
    check_policy(r, ref, c["xd"].shape[1], c["x"].dtype, c["adv"].astype(np.float64), c["old"].astype(np.float64),
                 None if c["refl"] is None else c["refl"].astype(np.float64), c["w"].astype(np.float64), c["T"],
                 c["kl"], c["ent"], **kw)


DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (2, 7), (5, 33), (4, 1000), (7, 4097), (3, 32000), (2, 70001),
                                 (2, 140000), (2, 270001)])
def test_policy_sizes(tsa, dtype, B, V):
    c = policy_case(np.random.default_rng(V), B, V, dtype, False, False, 0.1, 0.0)
    verify(c, call(tsa, c))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [5, 31, 257, 8192, 33001, 66000])
@pytest.mark.parametrize("mask,rowT,ent", [(True, False, 0.0), (False, True, 0.02), (True, True, 0.05)])
def test_policy_masks_temperatures_entropy(tsa, dtype, V, mask, rowT, ent):
    c = policy_case(np.random.default_rng(V + 1), 6, V, dtype, mask, rowT, 0.2 if ent else 0.0, ent)
    verify(c, call(tsa, c))


@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_loss_alone(tsa, dtype):
    c = policy_case(np.random.default_rng(3), 9, 5000, dtype, True, False, 0.1, 0.03)
    verify(c, call(tsa, c, grad=False), grad=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,stride", [(0, 1008), (1, 1008), (3, 1003), (0, 1001), (5, 2000)])
def test_policy_strides_and_alignment(tsa, dtype, offset, stride):
    c = policy_case(np.random.default_rng(4), 5, 1001, dtype, True, False, 0.1, 0.02)
    buf = torch.full((5 * stride + 64,), float("nan"), dtype=dtype, device=DEV)
    x = buf[offset:].as_strided((5, 1001), (stride, 1))
    x.copy_(c["x"])
    r = call(tsa, c, x)
    verify(c, r)
    # a gradient at another alignment, in guarded memory
    guard = torch.full((5 * 1002 + 64,), 7.0, dtype=dtype, device=DEV)
    g = guard[offset + 2:].as_strided((5, 1001), (1002, 1))
    r2 = call(tsa, c, x, grad=g)
    assert torch.equal(r2.grad, r.grad)
    rest = torch.ones_like(guard, dtype=torch.bool)
    rest[offset + 2:].as_strided((5, 1001), (1002, 1)).fill_(False)
    assert torch.all(guard[rest] == 7.0)
    # over the logits themselves
    r3 = call(tsa, c, x, grad=x)
    assert r3.grad is x and torch.equal(x, r.grad) and torch.equal(r3.row_loss, r.row_loss)
    left = torch.ones_like(buf, dtype=torch.bool)
    left[offset:].as_strided((5, 1001), (stride, 1)).fill_(False)
    assert torch.all(torch.isnan(buf[left]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [100, 40000, 300000])
def test_policy_rows_that_do_not_count(tsa, dtype, V):
    rng = np.random.default_rng(8)
    c = policy_case(rng, 6, V, dtype, True, False, 0.1, 0.02)
    c["w"][0] = 0.0
    c["x"][0] = float("nan")
    c["tok"][1] = -1
    c["x"][1] = float("inf")
    c["tok"][2] = V
    c["allowed"][3] = False  # the row allows nothing
    c["allowed"][4, c["tok"][4]] = False  # it excludes its token
    c["xd"] = c["x"].double().numpy()
    r = call(tsa, c)
    verify(c, r)
    g = r.grad.cpu()
    assert torch.all(g[:5] == 0) and torch.all(r.row_loss.cpu()[:5] == 0)
    assert r.logprob[4].item() == float("-inf") and torch.isnan(r.logprob[3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [64, 20000, 300000])
def test_policy_special_logits(tsa, dtype, V):
    rng = np.random.default_rng(9)
    c = policy_case(rng, 5, V, dtype, False, False, 0.0, 0.01)
    lowest = torch.finfo(dtype).min
    keep = (c["tok"][0] + 1) % V
    c["x"][0, keep] = float("nan")  # counts as -inf
    c["x"][1] = lowest  # a row of the type's lowest value is uniform
    c["x"][2, : V // 2] = lowest
    c["x"][3, V // 3:] = float("-inf")
    c["tok"][2], c["tok"][3] = V - 1, 0
    c["xd"] = c["x"].double().numpy()
    lp = losses.policy_loss(c["xd"], c["tok"], np.zeros(5), c["adv"])["logprob"]
    c["old"] = (lp + 0.1).astype(np.float32)
    verify(c, call(tsa, c))
    # +inf makes its row NaN, and leaves the others alone
    c["x"][4, 5] = float("inf")
    r = call(tsa, c)
    assert torch.isnan(r.loss) and torch.isnan(r.row_loss[4]) and torch.isnan(r.grad[4]).all()
    assert torch.isfinite(r.grad[:4].float()).all()


def test_policy_zero_advantage_and_overflowing_ratio(tsa):
    x = torch.zeros(3, 16, device=DEV)
    tok = torch.zeros(3, dtype=torch.int64, device=DEV)
    old = f32([-200.0, -200.0, -200.0])
    r = tsa.policy_loss(x, tok, old, f32([0.0, 1.0, -1.0]))
    assert r.row_loss[0].item() == 0.0 and r.row_loss[1].item() == pytest.approx(-1.2)
    assert r.row_loss[2].item() == float("inf") and torch.all(r.grad[:2] == 0)


def test_policy_far_from_zero(tsa):
    # rows shifted by a constant have the same loss and gradient up to the logits' own rounding
    rng = np.random.default_rng(10)
    for shift in (1e4, -1e4):
        c = policy_case(rng, 4, 3000, torch.float32, False, False, 0.1, 0.02)
        c["x"] = c["x"] + shift
        c["xd"] = c["x"].double().numpy()
        lp = losses.policy_loss(c["xd"], c["tok"], np.zeros(4), c["adv"])["logprob"]
        c["old"], c["refl"] = (lp + 0.1).astype(np.float32), (lp - 0.2).astype(np.float32)
        verify(c, call(tsa, c))


def test_policy_equal_calls_equal_bits_and_streams(tsa):
    c = policy_case(np.random.default_rng(11), 300, 9001, torch.bfloat16, True, True, 0.1, 0.02)
    a = call(tsa, c)
    side = torch.cuda.Stream()
    x = c["x"].to(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call(tsa, c, x)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("dtype,B,V", [(torch.bfloat16, 400, 33000), (torch.float32, 150, 40000),
                                       (torch.float16, 2500, 301), (torch.bfloat16, 130, 140000)])
def test_policy_many_rows_with_gaps(tsa, grad, dtype, B, V):
    # more rows than run at once, with single, short and long runs of skipped rows among them; the
    # rows repeat a few reference rows, so that the definition is evaluated once for each
    rng = np.random.default_rng(B)
    c = policy_case(rng, 5, V, dtype, False, False, 0.1, 0.02)
    ref = reference(c)
    pick = rng.integers(0, 5, B)
    w = rng.random(B).astype(np.float32) + 0.1
    skip = rng.random(B) < 0.2
    skip[B // 3:B // 2] = True
    skip[-3:] = True
    w[skip] = 0.0
    g = lambda a: f32(np.asarray(a)[pick])  # noqa: E731
    x = c["x"].to(DEV)[torch.from_numpy(pick).to(DEV)]
    x[torch.from_numpy(skip).to(DEV)] = float("nan")
    r = tsa.policy_loss(x, torch.from_numpy(c["tok"][pick]).to(DEV), g(c["old"]), g(c["adv"]), ref_logprob=g(c["refl"]),
                        weight=f32(w), clip_low=0.2, clip_high=0.3, kl_coef=0.1, entropy_coef=0.02,
                        return_entropy=True, grad=grad)
    live = ~skip
    one = tsa.policy_loss(c["x"].to(DEV), torch.from_numpy(c["tok"]).to(DEV), f32(c["old"]), f32(c["adv"]),
                          ref_logprob=f32(c["refl"]), weight=f32(np.ones(5)), clip_low=0.2, clip_high=0.3,
                          kl_coef=0.1, entropy_coef=0.02, return_entropy=True)
    tl = eps(V) + 3 * U * np.abs(ref["logprob"])
    check("logprob", r.logprob, np.where(live, ref["logprob"][pick], 0.0), tl[pick])
    check("entropy", r.entropy, np.where(live, ref["entropy"][pick], 0.0), 4 * eps(V) * (1 + ref["entropy"][pick]))
    # the same row at another weight: the gradient is that many times the gradient at weight 1, each
    # rounded a few times in fp32 and once to its type
    if grad:
        base = one.grad.double()
        for b in range(B):
            got, want = r.grad[b].double(), base[pick[b]] * float(w[b])
            tol = want.abs() * (2 * OUT[dtype] + 2 ** -20) + 2 * TINY[dtype]
            assert torch.all((got - want).abs() <= tol + 2 ** -18 * want.abs().max()), b


def test_policy_empty_batch(tsa):
    z = torch.empty(0, 50, device=DEV)
    e = torch.empty(0, device=DEV)
    r = tsa.policy_loss(z, torch.empty(0, dtype=torch.int64, device=DEV), e, e)
    assert r.loss.item() == 0.0 and r.grad.shape == (0, 50)


def test_policy_gradient_against_differences(tsa):
    # central differences of the GPU's own loss in fp32 logits: the loss is known to a few 1e-7, a step of
    # 2^-6 gives a truncation error below |third derivative| 2^-12 / 6 (the loss is a softmax's, derivatives
    # of order 1) and a rounding error of 1e-6 / 2^-6
    c = policy_case(np.random.default_rng(12), 1, 12, torch.float32, True, False, 0.3, 0.1)
    c["w"][:] = 1.0
    c["old"] = (c["old"] * 0 + losses.policy_loss(c["xd"], c["tok"], np.zeros(1), c["adv"],
                                                  allowed=c["allowed"])["logprob"] + 0.05).astype(np.float32)
    g = call(tsa, c).grad[0].cpu().numpy()
    for j in range(12):
        d = []
        for h in (2.0 ** -6, -2.0 ** -6):
            y = c["x"].clone()
            y[0, j] += h
            d.append(call(tsa, c, y.to(DEV)).loss.item())
        assert abs((d[0] - d[1]) * 32 - g[j]) < 5e-4, j


def pref_case(rng, start, V, dtype, ref, pad=0.2):
    N = start[-1]
    x, xd = rows(rng, N, V, dtype, 2.0)
    tok = rng.integers(0, V, N)
    w = np.where(rng.random(N) < pad, 0.0, 1.0).astype(np.float32)
    refl = None
    if ref:
        lp = losses.preference_loss(xd, tok, [0, N, N])["logprob"]
        refl = (lp + 0.3 * rng.standard_normal(N)).astype(np.float32)
    return dict(x=x, xd=xd, tok=tok, w=w, refl=refl, start=start)


def check_preference(r, c, V, dtype, beta, smooth, margin, average, T=1.0, grad=True):
    f = np.float64
    ref = losses.preference_loss(c["xd"], c["tok"], c["start"], c["w"], c["refl"], f(np.float32(beta)),
                                 f(np.float32(smooth)), f(np.float32(margin)), average, f(np.float32(T)))
    lp = np.where(np.isfinite(ref["logprob"]), ref["logprob"], 0.0)
    tl = eps(V) + 3 * U * np.abs(lp)
    check("logprob", r.logprob, ref["logprob"], tl)
    S = len(c["start"]) - 1
    tR = np.zeros(S)
    for s in range(S):
        a, b = c["start"][s], c["start"][s + 1]
        n = (c["w"][a:b] != 0).sum() if average else 1
        tR[s] = (np.abs(c["w"][a:b]) * tl[a:b]).sum() / max(n, 1)
    check("reward", r.reward, ref["reward"], beta * tR + 2 * U * np.abs(ref["reward"]) + 1e-30)
    P = S // 2
    th = beta * (tR[:P] + tR[P:]) + 2 * U * (np.abs(ref["reward"][:P]) + np.abs(ref["reward"][P:]) + abs(margin))
    check("pair_loss", r.pair_loss, ref["pair_loss"], th + 8 * U * (1 + ref["pair_loss"]))
    check("loss", r.loss.reshape(1), [ref["loss"]], th.mean() + 8 * U * (1 + ref["loss"]) if P else 0.0)
    if grad:
        # a row's coefficient moves with h by at most itself (logistic), plus its own roundings
        tc = np.zeros(c["start"][-1])
        for s in range(S):
            tc[c["start"][s]:c["start"][s + 1]] = beta / P * (th[s % P] + 16 * U)
        g = np.abs(ref["grad"])
        Tb = T if T > 0 else 1.0
        hot = np.zeros_like(g)
        ok = (c["tok"] >= 0) & (c["tok"] < V)
        hot[np.arange(len(ok))[ok], c["tok"][ok]] = 1.0
        small = (np.abs(ref["coef"]) * 4 * eps(V) + tc)[:, None] / Tb
        p = g / np.maximum(np.abs(ref["coef"])[:, None], 1e-300) * Tb
        live = (ref["coef"] != 0)[:, None]
        check("grad", r.grad, ref["grad"],
              g * (2 * OUT[dtype] + 8 * eps(V)) + live * small * np.minimum(1.0, p + hot) + TINY[dtype])


def call_pref(tsa, c, x=None, **kw):
    x = c["x"].to(DEV) if x is None else x
    return tsa.preference_loss(x, torch.from_numpy(np.asarray(c["tok"], np.int64)).to(DEV),
                               torch.tensor(c["start"], dtype=torch.int64, device=DEV), weight=f32(c["w"]),
                               ref_logprob=None if c["refl"] is None else f32(c["refl"]), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,lengths", [(1, [1, 2]), (9, [1, 1]), (100, [3, 0, 1, 7]), (5003, [4, 9, 1, 2, 6, 3]),
                                       (33000, [2, 5]), (140001, [1, 3]), (300000, [2, 1])])
@pytest.mark.parametrize("smooth,margin,average", [(0.1, 0.0, False), (0.0, 0.4, True)])
def test_preference_sizes(tsa, dtype, V, lengths, smooth, margin, average):
    start = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    c = pref_case(np.random.default_rng(V), start, V, dtype, not average)
    r = call_pref(tsa, c, beta=0.5, label_smoothing=smooth, margin=margin, average=average)
    check_preference(r, c, V, dtype, 0.5, smooth, margin, average)


def test_preference_many_rows_and_temperature(tsa):
    rng = np.random.default_rng(21)
    start = np.concatenate([[0], np.cumsum(rng.integers(1, 60, 24))]).tolist()
    c = pref_case(rng, start, 777, torch.bfloat16, True)
    check_preference(call_pref(tsa, c, temperature=0.7), c, 777, torch.bfloat16, 0.1, 0.0, 0.0, False, 0.7)


def test_preference_in_place_loss_alone_and_skipped_rows(tsa):
    rng = np.random.default_rng(22)
    c = pref_case(rng, [2, 6, 9, 9, 13], 3001, torch.float16, True)  # rows 0, 1 belong to no sequence
    c["xd"], c["x"] = c["xd"], c["x"]
    c["w"][3] = 0.0
    c["x"][3] = float("nan")
    c["tok"][7] = -1
    c["x"][10, c["tok"][10]] = float("-inf")
    c["w"][10] = 1.0
    c["xd"] = c["x"].double().numpy()
    r = call_pref(tsa, c, beta=0.3)
    check_preference(r, c, 3001, torch.float16, 0.3, 0.0, 0.0, False)
    assert torch.all(r.grad[[0, 1, 3, 7, 10]] == 0)
    alone = call_pref(tsa, c, beta=0.3, grad=False)
    assert alone.grad is None and torch.equal(alone.pair_loss, r.pair_loss)
    x = c["x"].to(DEV)
    inplace = call_pref(tsa, c, x, beta=0.3, grad=x)
    assert inplace.grad is x and torch.equal(x, r.grad)


def test_preference_extremes(tsa):
    # log-ratios that saturate the logistic: the loss is linear on one side and 0 on the other
    x = torch.zeros(2, 8, device=DEV)
    x[0, 0], x[1, 0] = 50.0, -50.0
    tok = torch.zeros(2, dtype=torch.int64, device=DEV)
    start = torch.tensor([0, 1, 2], device=DEV)
    r = tsa.preference_loss(x, tok, start, beta=4.0)
    assert r.loss.item() == 0.0 or r.loss.item() < 1e-30
    r = tsa.preference_loss(x, tok, torch.tensor([0, 1, 2], device=DEV), beta=-4.0)
    assert r.loss.item() == pytest.approx(4.0 * (50.0 + np.log(7.0)), rel=1e-6)


def test_preference_no_pairs(tsa):
    r = tsa.preference_loss(torch.zeros(3, 10, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV),
                            torch.zeros(1, dtype=torch.int64, device=DEV))
    assert r.loss.item() == 0.0 and torch.all(r.grad == 0)


def test_preference_gradient_against_differences(tsa):
    c = pref_case(np.random.default_rng(23), [0, 2, 3], 6, torch.float32, True, pad=0.0)
    g = call_pref(tsa, c, beta=1.0).grad.cpu().numpy()
    for i in range(3):
        for j in range(6):
            d = []
            for h in (2.0 ** -6, -2.0 ** -6):
                y = c["x"].clone()
                y[i, j] += h
                d.append(call_pref(tsa, c, y.to(DEV), beta=1.0).loss.item())
            assert abs((d[0] - d[1]) * 32 - g[i, j]) < 5e-4


def test_refusals(tsa):
    x = torch.zeros(2, 10, device=DEV)
    tok, v = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(2, device=DEV)
    for kw in (dict(tokens=tok.int()), dict(old_logprob=v.double()), dict(advantage=v[:1]),
               dict(weight=torch.zeros(2)), dict(grad=torch.zeros(2, 9, device=DEV)),
               dict(grad=torch.zeros(2, 10, device=DEV, dtype=torch.float16)),
               dict(bitmask=torch.zeros(2, 1, device=DEV))):
        a = dict(tokens=tok, old_logprob=v, advantage=v, **{k: kw[k] for k in kw if k in ("weight", "grad", "bitmask")})
        a.update({k: kw[k] for k in kw if k in ("tokens", "old_logprob", "advantage")})
        with pytest.raises(ValueError):
            tsa.policy_loss(x, **a)
    with pytest.raises(tsa.TSAError):
        tsa.policy_loss(x, tok, v, v, clip_low=-0.1)
    with pytest.raises(tsa.TSAError):
        tsa.policy_loss(x, tok, v, v, kl_coef=float("nan"))
    with pytest.raises(ValueError):
        tsa.preference_loss(x, tok, torch.tensor([0, 1], device=DEV))
    with pytest.raises(ValueError):
        tsa.preference_loss(x, tok, torch.tensor([0, 1, 2]))
    with pytest.raises(tsa.TSAError):
        tsa.preference_loss(x, tok, torch.tensor([0, 1, 2], device=DEV), label_smoothing=1.5)


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
@pytest.mark.parametrize("row,inf_in", [(1, 0), (6, 2)])
def test_preference_infinite_reference(tsa, row, inf_in, smooth, average):
    # a token that the reference's mask excludes has ref -inf: the log-ratio is +inf, the pair's loss by the formula 0 or
    # +inf, and the gradient that of a saturated logistic, as a far finite reference has it
    c = pref_case(np.random.default_rng(30), [0, 3, 5, 9, 11], 2003, torch.float32, True, pad=0.0)
    far = dict(c, refl=c["refl"].copy())
    far["refl"][row] = -1e6  # h is 1e5 and more: the logistic of it is 0 or 1 in 64 bits too
    c["refl"][row] = -np.inf
    kw = dict(beta=0.5, label_smoothing=smooth, average=average)
    r, f = call_pref(tsa, c, **kw), call_pref(tsa, far, **kw)
    check_preference(f, far, 2003, torch.float32, 0.5, smooth, 0.0, average)
    assert r.reward[inf_in].item() == float("inf")
    assert r.pair_loss[0].item() == (0.0 if inf_in == 0 and smooth == 0.0 else float("inf"))
    assert r.loss.item() == (float("inf") if r.pair_loss[0].item() else r.pair_loss[1].item() / 2)
    others = [s for s in range(4) if s != inf_in]
    assert torch.equal(r.reward[others], f.reward[others]) and torch.equal(r.pair_loss[1], f.pair_loss[1])
    assert torch.equal(r.grad, f.grad) and torch.equal(r.logprob, f.logprob)


def test_preference_smoothing_of_one(tsa):
    # label_smoothing 1 leaves the rejected answer's term alone: 0 where that answer is infinitely preferred
    x, tok = torch.zeros(2, 8, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    start = torch.tensor([0, 1, 2], device=DEV)
    r = tsa.preference_loss(x, tok, start, ref_logprob=f32([0.0, -np.inf]), label_smoothing=1.0)
    assert r.loss.item() == 0.0 and r.pair_loss[0].item() == 0.0 and torch.all(r.grad == 0)


@pytest.mark.parametrize("V", [700, 300001])
def test_policy_without_a_kl_coefficient_has_no_kl_term(tsa, V):
    # kl_coef 0 beside a reference that excludes the token, or holds it far more likely than exp can tell
    c = policy_case(np.random.default_rng(31), 4, V, torch.float32, False, False, 0.0, 0.02)
    want = call(tsa, c)
    ref = f32([-np.inf, 1000.0, -0.5, np.inf])
    for kw in ({}, {"grad": False}):
        got = call(tsa, c, ref_logprob=ref, kl_coef=0.0, **kw)
        for name in ("loss", "row_loss", "logprob", "entropy"):
            assert torch.equal(getattr(got, name), getattr(want, name)) or kw, name
        assert torch.isfinite(got.loss) and torch.isfinite(got.row_loss).all()
        assert kw or torch.equal(got.grad, want.grad)


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_a_gradient_over_the_logits_is_seen_by_autograd(tsa, loss):
    tok, v = torch.zeros(2, dtype=torch.int64, device=DEV), torch.ones(2, device=DEV)

    def run(y, grad):
        if loss == "policy":
            return tsa.policy_loss(y, tok, -v, v, grad=grad)
        return tsa.preference_loss(y, tok, torch.tensor([0, 1, 2], device=DEV), grad=grad)

    x = torch.randn(2, 64, device=DEV, requires_grad=True)
    y = torch.tanh(x)  # its backward needs y as it was
    r = run(y, y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(r.grad)
    # a product does not need its output: the gradient goes on
    w = torch.randn(64, 80, device=DEV)
    y = x @ w
    want = run(y.detach(), True).grad
    r = run(y, y)
    y.backward(r.grad.detach())
    assert torch.equal(r.grad, want) and torch.allclose(x.grad, want @ w.t(), rtol=1e-4, atol=1e-6)
    other = torch.empty_like(want)
    before = other._version
    run(y.detach(), other)
    assert other._version > before
    with torch.inference_mode():
        z = torch.randn(2, 64, device=DEV)
        run(z, z)
    run(z, z)  # an inference tensor has no version


@pytest.mark.parametrize("dtype,B,V,grad", [(torch.bfloat16, 40, 9001, True), (torch.float32, 9, 5000, False),
                                            (torch.float16, 3, 300000, True)])
def test_policy_replays_in_a_graph(tsa, dtype, B, V, grad):
    cases = [policy_case(np.random.default_rng(s), B, V, dtype, True, True, 0.1, 0.02) for s in (40, 41)]
    keys = ("x", "tok", "old", "adv", "refl", "w", "T")
    put = lambda c, k: (c[k] if torch.is_tensor(c[k]) else torch.from_numpy(np.asarray(c[k]))).to(DEV)  # noqa: E731
    a = {k: put(cases[0], k) for k in keys}
    a["mask"] = pack(cases[0]["allowed"])

    def run():
        return tsa.policy_loss(a["x"], a["tok"], a["old"], a["adv"], ref_logprob=a["refl"], weight=a["w"], kl_coef=0.1,
                               entropy_coef=0.02, temperature=a["T"], bitmask=a["mask"], return_entropy=True, grad=grad)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run()
    for c in cases[::-1]:
        for k in keys:
            a[k].copy_(put(c, k))
        a["mask"].copy_(pack(c["allowed"]))
        g.replay()
        for p, q in zip(r, run()):
            assert p is q is None or torch.equal(p, q)


@pytest.mark.parametrize("in_place", [True, False])
def test_preference_replays_in_a_graph(tsa, in_place):
    start = [0, 4, 5, 11, 14]
    cases = [pref_case(np.random.default_rng(s), start, 4001, torch.bfloat16, True) for s in (42, 43)]
    keys = ("x", "tok", "w", "refl")
    put = lambda c, k: (c[k] if torch.is_tensor(c[k]) else torch.from_numpy(np.asarray(c[k]))).to(DEV)  # noqa: E731
    a = {k: put(cases[0], k) for k in keys}
    st = torch.tensor(start, device=DEV)

    def run(x):
        return tsa.preference_loss(x, a["tok"], st, weight=a["w"], ref_logprob=a["refl"], grad=x if in_place else True)

    run(a["x"].clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run(a["x"])
    for c in cases[::-1]:
        for k in keys:
            a[k].copy_(put(c, k))
        want = run(a["x"].clone())
        g.replay()
        for p, q in zip(r, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_log_probabilities_do_not_err_to_one_side(tsa, dtype):
    # A sequence's log-ratio adds up what its log-probabilities are off by on average.  With T = 1 that follows from two
    # things: ex2.approx is 5e-8 too small on average where it is not 1, and log2(e) as an fp32 number is 1.335e-8 of
    # itself too small, which makes a term at distance d from the row's largest d times that too large.  All else is
    # rounding to nearest, of which 4 standard errors may be left over these rows, and 1.5e-8 (an eighth of an fp32 ulp
    # of 1) where rows of like sums round alike.
    g = torch.Generator(device=DEV).manual_seed(50)
    V, N = 128256, 2048
    start, v = torch.tensor([0, N // 2, N], device=DEV), torch.zeros(N, device=DEV)
    off = {"preference": [], "policy": []}
    want = []
    for _ in range(8):
        rank = torch.randperm(V, generator=g, device=DEV).float().add_(1.0)
        x = torch.randn(N, V, generator=g, device=DEV).mul_(2.0).sub_(rank.log_().mul_(1.1)).to(dtype)
        tok = torch.randint(0, V, (N,), generator=g, device=DEV)
        got = {"preference": tsa.preference_loss(x, tok, start, grad=False).logprob,
               "policy": tsa.policy_loss(x, tok, v, v).logprob}
        for a in range(0, N, 512):
            d = x[a:a + 512].double()
            d -= d.amax(1, keepdim=True)
            e = d.exp()
            Z = e.sum(1)
            lp = d.gather(1, tok[a:a + 512, None])[:, 0] - Z.log()
            want.append(5e-8 * (1 - 1 / Z) + 1.335e-8 * (e * d).sum(1) / Z)
            for k in off:
                off[k].append(got[k][a:a + 512].double() - lp)
    want = torch.cat(want).mean().item()
    for k, o in off.items():
        o = torch.cat(o)
        left = 1.5e-8 + 4 * o.std().item() / len(o) ** 0.5
        assert abs(o.mean().item() - want) <= left, (k, o.mean().item(), want, left)
