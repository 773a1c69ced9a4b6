"""lm_head_cross_entropy on the GPU against float64.

Tolerances, with u = 2^-24.  A score is off by at most d = H 2^-23 sum |h w| + 2^-21 max(cap, |z|) (fp32 sums that the
tensor cores cut, the bias, the cap), and so is the log-sum-exp but for its own rounding, e = (132 + V / 128) u.
exp(z - l) is then off by 2 d + e + 4 u of itself, the slope of the cap by 4 (d + 2^-21 cap) / cap, and G is rounded
to bf16 (2^-8 of itself).  Products over K terms add K 2^-23 of the sum of absolute terms, gradients are rounded to
bf16 again."""
import pytest
import torch

from oracle import head

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def tsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import top_sampling_apply_gb300 as lib

    lib.load_library()
    return lib


def make(seed, M, V, H, bias=False, skip=0.0, weighted=False, pad=0, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    hb = torch.full((M, H + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wb = torch.full((V, H + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    h, w = hb[:, :H], wb[:, :H]
    h.copy_(torch.randn(M, H, generator=g, device=DEV))
    w.copy_(torch.randn(V, H, generator=g, device=DEV) * (scale / H ** 0.5))
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    out = torch.rand(M, generator=g, device=DEV) < skip
    t[out] = -100
    h[out] = float("nan")  # what a skipped row holds is not used
    return dict(h=h, w=w, t=t, b=torch.randn(V, generator=g, device=DEV) if bias else None,
                row_weight=torch.rand(M, generator=g, device=DEV) * 0.1 if weighted else None)


def near(got, want, tol, name):
    got = got.double()
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert (err <= tol).all(), (name, (err / tol.clamp(min=1e-300)).max().item())


def check(c, r, cap=0.0, z_loss=0.0):
    h, w, t = c["h"], c["w"], c["t"]
    V, H = w.shape
    x = head.cross_entropy(h, w, t, c["b"], cap, c["row_weight"], z_loss)
    live, k = x["live"], x["c"].abs()
    a, aw = torch.where(live[:, None], h.double().abs(), 0.0), w.double().abs()
    # entries of -inf have the exact exponential 0, and no part in any rounding
    z = torch.where(torch.isinf(x["z"]), 0.0, x["z"])
    d = H * 2.0 ** -23 * (a @ aw.T).amax(1) + 2.0 ** -21 * z.abs().amax(1).clamp(min=cap)
    e = (132 + V / 128) * U + 3 * U * x["lse"].abs()
    l = x["lse"].abs()
    tol_l = torch.where(live, d + e, 0.0)
    near(r.lse, x["lse"], tol_l, "lse")
    tol_row = torch.where(live, 2 * d + e + abs(z_loss) * (2 * l + 1) * (d + e) + 4 * U * x["row"].abs(), 0.0)
    near(r.row_loss, x["row"], tol_row, "row")
    near(r.loss, x["loss"], (k * (tol_row + 2 * U * x["row"].abs())).sum() + U * x["loss"].abs(), "loss")
    p = torch.exp(x["z"] - torch.where(live, x["lse"], 0.0)[:, None]) * live[:, None]
    dg = (k * (1 + 2 * abs(z_loss) * (l + 1)) * (2 * d + e + 8 * U + 4 * abs(z_loss) * (d + e)))[:, None] * p
    if cap > 0:
        dg = dg + 4 * (d / cap + 2.0 ** -21)[:, None] * (k[:, None] * p + torch.where(
            torch.arange(V, device=DEV) == t[:, None], k[:, None], 0.0))
    dg = dg + 4 * U * x["G"].abs()
    if r.grad_bias is not None:
        n = int(live.sum())
        near(r.grad_bias, x["db"], dg.sum(0) + (n + 8) * U * x["G"].abs().sum(0) + 1e-38, "db")
    dg = dg + 2.0 ** -8 * (x["G"].abs() + dg)
    g = x["G"].abs() + dg
    if r.grad_hidden is not None:
        tol = dg @ aw + V * 2.0 ** -23 * (g @ aw)
        near(r.grad_hidden, x["dh"], tol + 2.0 ** -8 * (x["dh"].abs() + tol), "dh")
    if r.grad_weight is not None:
        tol = dg.T @ a + len(t) * 2.0 ** -23 * (g.T @ a)
        near(r.grad_weight, x["dw"], tol + 2.0 ** -8 * (x["dw"].abs() + tol), "dw")
    return x


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 100, 128, 129, 300])
@pytest.mark.parametrize("V,H", [(1, 8), (33, 64), (256, 136), (1000, 72), (4099, 520)])
def test_sizes(tsa, M, V, H):
    c = make(M * 7 + V, M, V, H)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]))


@pytest.mark.parametrize("M", [3, 20, 90, 260])
@pytest.mark.parametrize("V,H", [(257, 128), (8001, 264)])
@pytest.mark.parametrize("cap,z_loss", [(0.0, 0.0), (5.0, 1e-3), (30.0, 0.0)])
def test_bias_cap_weights_skips_strides(tsa, M, V, H, cap, z_loss):
    c = make(M + V, M, V, H, bias=True, skip=0.3, weighted=True, pad=24)
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap, row_weight=c["row_weight"],
                                  z_loss=z_loss)
    check(c, r, cap, z_loss)
    c["row_weight"] = None
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap, z_loss=z_loss)
    check(c, r, cap, z_loss)


@pytest.mark.parametrize("M", [40, 200])
def test_given_gradients_and_parts(tsa, M):
    V, H = 700, 128
    c = make(M, M, V, H, bias=True, skip=0.2)
    hb = torch.full((M, H + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    wb = torch.full((V, H + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    db = torch.full((V,), 7.0, device=DEV)
    whole = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], grad_hidden=hb[:, :H], grad_weight=wb[:, :H],
                                  grad_bias=db)
    assert r.grad_bias is db and db._version > 0 and wb._version > 0
    check(c, r)
    assert (hb[:, H:] == 7).all() and (wb[:, H:] == 7).all()
    for k in range(8):  # any of the gradients
        r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], grad_hidden=bool(k & 1),
                                      grad_weight=bool(k & 2), grad_bias=bool(k & 4))
        for on, name in ((k & 1, "grad_hidden"), (k & 2, "grad_weight"), (k & 4, "grad_bias")):
            a, b = getattr(r, name), getattr(whole, name)
            assert (a is None) if not on else torch.equal(a, b), (k, name)
        assert torch.equal(r.loss, whole.loss) and torch.equal(r.row_loss, whole.row_loss)


def test_no_row_counts(tsa):
    c = make(1, 50, 300, 64, bias=True)
    c["t"][:25], c["t"][25:] = -1, 300
    c["h"].fill_(float("nan"))
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    for x in r:
        assert (x == 0).all()
    r = tsa.lm_head_cross_entropy(c["h"][:0], c["w"], c["t"][:0], bias=c["b"])
    assert r.grad_hidden.shape == (0, 64) and (r.grad_weight == 0).all() and (r.grad_bias == 0).all() and r.loss == 0


def test_zero_weights_skip(tsa):
    c = make(2, 70, 500, 64, weighted=True)
    c["row_weight"][::3] = 0.0
    c["h"][::3] = float("inf")
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], row_weight=c["row_weight"]))


@pytest.mark.parametrize("M", [4, 140])
def test_scores_far_apart_and_infinite(tsa, M):
    c = make(M, M, 2000, 64, bias=True)
    c["b"][5], c["b"][6:900] = 3e4, -3e4
    c["t"][0] = 5
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"]))
    c["b"][5:900] = float("-inf")  # excluded entries
    c["t"] = c["t"] % 5
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    x = check(c, r)
    assert (x["G"][:, 5:900] == 0).all() and (r.grad_weight[5:900] == 0).all() and (r.grad_bias[5:900] == 0).all()
    c["b"][7] = float("nan")  # counts as -inf
    again = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    assert all(torch.equal(p, q) for p, q in zip(r, again))
    c["b"][3] = float("inf")
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    assert (r.lse == float("inf")).all() and torch.isnan(r.row_loss).all() and torch.isnan(r.loss)
    assert torch.isnan(r.grad_hidden).all() and torch.isnan(r.grad_weight[3]).all()


def test_repeats_on_another_stream(tsa):
    c = make(3, 200, 3000, 256, bias=True, skip=0.1)
    a = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], z_loss=1e-4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], z_loss=1e-4)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and tsa.device_status() == 0


@pytest.mark.parametrize("M", [20, 150, 1000])
def test_captured_and_replayed_on_new_inputs(tsa, M):
    c, d = make(3, M, 3000, 256, skip=0.1), make(4, M, 3000, 256, skip=0.5)
    graph = torch.cuda.CUDAGraph()
    tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"])
    for x in (c, d):
        want = tsa.lm_head_cross_entropy(x["h"], x["w"], x["t"])
        for n in ("h", "w", "t"):
            c[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(r[:5], want[:5]))


def test_more_rows_than_one_pass(tsa):
    c = make(5, 8192 + 300, 600, 64, skip=0.01)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]))


def test_several_pieces_of_the_vocabulary(tsa):
    c = make(5, 8192 + 300, 9001, 64, bias=True, skip=0.01)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"]))


def test_most_rows(tsa):
    c = make(9, 65536, 130, 64, skip=0.02)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]))
    with pytest.raises(tsa.TSAError):
        tsa.lm_head_cross_entropy(torch.cat([c["h"], c["h"][:1]]), c["w"], torch.cat([c["t"], c["t"][:1]]))


def test_weight_of_more_elements_than_32_bits_count(tsa):
    M, V, H = 40, 560_000, 4096
    g = torch.Generator(device=DEV).manual_seed(0)
    w = torch.empty(V, H, dtype=torch.bfloat16, device=DEV).normal_(0.0, 0.05, generator=g)
    h = torch.randn(M, H, generator=g, device=DEV).bfloat16()
    t = torch.randint(V - 5000, V, (M,), generator=g, device=DEV)
    assert w.numel() > 2 ** 31
    r = tsa.lm_head_cross_entropy(h, w, t)
    z = torch.cat([h.double() @ w[i:i + 70_000].double().T for i in range(0, V, 70_000)], 1)
    lse = torch.logsumexp(z, -1)
    G = torch.exp(z - lse[:, None]) / M
    G[torch.arange(M, device=DEV), t] -= 1.0 / M
    assert ((r.lse.double() - lse).abs() < 1e-4).all()
    # bf16 G and results: 2^-8 of the sums of absolute terms
    last = slice(V - 6000, V)
    want, bound = G[:, last].T @ h.double(), G[:, last].abs().T @ h.double().abs()
    assert ((r.grad_weight[last].double() - want).abs() <= 2.0 ** -7 * bound + 1e-30).all()
    dh = sum(G[:, i:i + 70_000] @ w[i:i + 70_000].double() for i in range(0, V, 70_000))
    assert (r.grad_hidden.double() - dh).norm() / dh.norm() < 2.0 ** -8


def test_calls_at_once_on_two_streams(tsa):
    cs = [make(20 + i, M, 5000, 512, skip=0.1) for i, M in enumerate((70, 300, 1100))]
    want = [tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a[:5], b[:5]))
    assert tsa.device_status() == 0


def test_large(tsa):
    c = make(6, 700, 20001, 1024, bias=True, skip=0.2)
    x = check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"]))
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    # two roundings to bf16, each at most 2^-8 and 2^-9 / sqrt(3) of it in the mean
    for got, want in ((r.grad_hidden, x["dh"]), (r.grad_weight, x["dw"])):
        assert (got.double() - want).norm() / want.norm() < 2.0 ** -8


def test_is_lm_head_logprob_and_policy_gradient(tsa):
    """The row's loss is the negative log-probability, and the gradient of the scores that of a policy loss."""
    c = make(8, 64, 1000, 128)
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"])
    assert torch.equal(r.row_loss, -tsa.lm_head_logprob(c["h"], c["w"], c["t"]))
    z = c["h"].float() @ c["w"].float().T
    lp = tsa.selective_log_softmax(z, c["t"])
    g = tsa.policy_loss(z, c["t"], lp, torch.ones(64, device=DEV)).grad  # at ratio 1: -grad ln p
    want = g.double() @ c["w"].double()
    assert (r.grad_hidden.double() - want).norm() / want.norm() < 2.0 ** -8


def test_training_step_together(tsa):
    """Norm, cross entropy, the norm's backward pass and a step, with gradients against differences of the loss."""
    g = torch.Generator(device=DEV).manual_seed(0)
    M, V, H = 96, 800, 128
    x = torch.randn(M, H, generator=g, device=DEV).bfloat16()
    gain = (torch.rand(H, generator=g, device=DEV) + 0.5)
    w = (torch.randn(V, H, generator=g, device=DEV) * 0.2).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    t[::5] = -1
    dw = torch.zeros_like(w)
    plan = tsa.adamw_plan([w], [dw], *tsa.adamw_state([w]))
    n = tsa.rms_norm(x, gain)
    r = tsa.lm_head_cross_entropy(n.out, w, t, grad_weight=dw)
    dx, dgain = tsa.rms_norm_backward(r.grad_hidden, x, gain, n.rstd)

    def loss(x, gain, w):
        return head.cross_entropy(head.rms_norm(x, gain, 1e-6)[0], w, t)["loss"]

    for a, b in ((x, dx), (gain, dgain), (w, r.grad_weight)):
        d = b.double() / b.double().norm()  # along the gradient: its own norm
        f = lambda k: loss(*(y.double() + k * d if y is a else y for y in (x, gain, w)))  # noqa: E731
        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        # bf16 hidden rows, G and gradients: three roundings of 2^-8 at most
        assert abs(slope / b.double().norm() - 1) < 3 * 2.0 ** -8
    before = w.clone()
    tsa.adamw_step(plan, 1, 1e-3, weight_decay=0.0, seed=1)
    assert not torch.equal(before, w)


def test_refusals(tsa):
    c = make(1, 4, 64, 32, bias=True)
    h, w, t, b = c["h"], c["w"], c["t"], c["b"]
    f = tsa.lm_head_cross_entropy
    for call in (lambda: f(h.float(), w, t), lambda: f(h, w.half(), t), lambda: f(h, w, t.int()), lambda: f(h, w, t[:2]),
                 lambda: f(h, w[:, :16], t), lambda: f(h, w, t, bias=b[:5]), lambda: f(h, w, t, row_weight=b),
                 lambda: f(h, w, t, grad_hidden=w), lambda: f(h, w, t, grad_weight=w.float()),
                 lambda: f(h, w, t, grad_bias=b), lambda: f(h.t(), w, t)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(h, w, t, softcap=-1.0), lambda: f(h, w, t, z_loss=float("nan")),
                 lambda: f(h[:, :12].contiguous(), w[:, :12].contiguous(), t)):
        with pytest.raises(tsa.TSAError):
            call()


@pytest.mark.parametrize("M", [4, 140, 1000])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_a_row_without_a_finite_score(tsa, M, cap):
    """It has an lse of -inf, a loss of NaN and a gradient of NaN; a skipped row like it has nothing of that."""
    c = make(M, M, 700, 72, bias=True)
    c["h"][1], c["h"][2], c["t"][2] = float("nan"), float("nan"), -1
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap)
    assert r.lse[1] == float("-inf") and torch.isnan(r.row_loss[1]) and torch.isnan(r.loss)
    assert torch.isnan(r.grad_hidden[1]).all() and torch.isnan(r.grad_weight).all() and torch.isnan(r.grad_bias).all()
    others = torch.arange(M, device=DEV) != 1
    assert torch.isfinite(r.grad_hidden[others]).all() and torch.isfinite(r.row_loss[others]).all()
    assert r.lse[2] == 0 and r.row_loss[2] == 0 and (r.grad_hidden[2] == 0).all()


@pytest.mark.parametrize("M", [4, 140, 1000])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_a_score_of_nan_in_a_row_that_counts(tsa, M, cap):
    """It counts as -inf: no part in the row's loss, and none in the gradients of the other entries."""
    c = make(M, M, 700, 72, bias=True)
    c["b"][9] = float("nan")
    c["t"][c["t"] == 9] = 8
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap)
    keep = torch.arange(700, device=DEV) != 9
    d = dict(c, w=c["w"][keep], b=c["b"][keep], t=torch.where(c["t"] > 9, c["t"] - 1, c["t"]))
    assert (r.grad_weight[9] == 0).all() and r.grad_bias[9] == 0
    check(d, r._replace(grad_weight=r.grad_weight[keep], grad_bias=r.grad_bias[keep]), cap)


@pytest.mark.parametrize("M", [4, 140, 1000])
def test_no_row_counts_and_what_the_head_holds_is_not_finite(tsa, M):
    c = make(M, M, 700, 72, bias=True)
    c["t"].fill_(-1)
    c["b"][3], c["b"][4], c["b"][5], c["w"][6], c["w"][7] = (float(x) for x in ("inf", "-inf", "nan", "inf", "nan"))
    for cap in (0.0, 5.0):
        for x in tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap):
            assert (x == 0).all()


def fastest_ms(f, n=8):
    best = float("inf")
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


# two pieces of the vocabulary, whole, and one entry more: pairs of CTAs, single ones, one block of rows
@pytest.mark.parametrize("M,V", [(1000, 2 * 29_184), (300, 2 * 38_912), (100, 2 * 38_912)])
def test_a_last_piece_costs_what_it_holds(tsa, M, V):
    c, d = make(1, M, V, 1024), make(1, M, V + 1, 1024)
    whole, more = (fastest_ms(lambda: tsa.lm_head_cross_entropy(x["h"], x["w"], x["t"])) for x in (c, d))
    assert more < 1.5 * whole, (more, whole)


def live_rows(c, n):
    """All but n of the rows skipped, in no order, and what the skipped ones hold a NaN."""
    M = len(c["t"])
    out = torch.randperm(M, generator=torch.Generator().manual_seed(M + n))[n:].to(DEV)
    c["t"] = c["t"].clamp(min=0)
    c["t"][out], c["h"][out] = -1, float("nan")
    return c


def in_workspace_of(tsa, c, fill):
    """The call through the C entry, with a workspace that holds `fill` in every byte."""
    lib, (M, H), V = tsa.load_library(), c["h"].shape, c["w"].shape[0]
    dh, dw = torch.empty_like(c["h"]), torch.empty_like(c["w"])
    db, loss, row, lse = (torch.empty(n, device=DEV) for n in (V, 1, M, M))
    n = lib.tsa_lm_head_cross_entropy_workspace_bytes(M, H, V, 1, 1)
    ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
    st = lib.tsa_lm_head_cross_entropy(
        c["h"].data_ptr(), M, H, c["h"].stride(0), c["w"].data_ptr(), V, c["w"].stride(0), c["b"].data_ptr(), 0.0,
        c["t"].data_ptr(), None, 0.0, loss.data_ptr(), row.data_ptr(), lse.data_ptr(), dh.data_ptr(), dh.stride(0),
        dw.data_ptr(), dw.stride(0), db.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    return loss, row, lse, dh, dw, db


# one block of rows, several, pairs; vocabularies of a part of a tile, of just over a piece, and of pieces and a half
@pytest.mark.parametrize("M,live,V", [(20, 20, 300), (20, 15, 65_600), (300, 200, 1000), (300, 300, 65_537),
                                      (1000, 1000, 29_185), (1100, 700, 29_000), (1100, 100, 1111), (9000, 8500, 6001)])
def test_workspaces_that_hold_anything(tsa, M, live, V):
    c = live_rows(make(M, M, V, 136, bias=True), live)
    a, b = in_workspace_of(tsa, c, 0xFF), in_workspace_of(tsa, c, 0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    check(c, tsa.CrossEntropy(a[0][0], *a[1:]))


# pairs of CTAs (rows from 897 on): 1, 2, 5, 8 and 9 blocks of 128 rows that count; widths of one and several K steps,
# column blocks and chunks of sums, multiples of 64 and not
@pytest.mark.parametrize("M,live", [(897, 897), (1023, 640), (1100, 1100), (1300, 130), (1100, 100)])
@pytest.mark.parametrize("V,H", [(3001, 136), (2500, 264), (4099, 520), (3000, 1088), (2001, 2056)])
@pytest.mark.parametrize("cap,z_loss", [(0.0, 0.0), (5.0, 1e-3)])
def test_pairs_of_ctas(tsa, M, live, V, H, cap, z_loss):
    c = live_rows(make(M + V, M, V, H, bias=True, weighted=True, pad=24), live)
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=cap, row_weight=c["row_weight"],
                                  z_loss=z_loss)
    check(c, r, cap, z_loss)
    c["row_weight"] = c["b"] = None
    r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], softcap=cap, z_loss=z_loss)
    check(c, r, cap, z_loss)


@pytest.mark.parametrize("M", [1, 100, 200, 1000])
@pytest.mark.parametrize("V,H", [(500, 1032), (700, 2056), (300, 5120), (400, 16376), (200, 16384)])
def test_wide_rows(tsa, M, V, H):
    c = make(M + H, M, V, H, bias=True, skip=0.1 if M > 1 else 0.0, pad=8)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], softcap=20.0, z_loss=1e-4), 20.0, 1e-4)


def test_each_gradient_of_pairs(tsa):
    c = live_rows(make(9, 1100, 3001, 328, bias=True), 900)
    whole = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"])
    check(c, whole)
    for k in range(8):
        r = tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"], bias=c["b"], grad_hidden=bool(k & 1),
                                      grad_weight=bool(k & 2), grad_bias=bool(k & 4))
        for on, name in ((k & 1, "grad_hidden"), (k & 2, "grad_weight"), (k & 4, "grad_bias")):
            a, b = getattr(r, name), getattr(whole, name)
            assert (a is None) if not on else torch.equal(a, b), (k, name)
        assert torch.equal(r.loss, whole.loss) and torch.equal(r.row_loss, whole.row_loss)


def test_sums_over_the_most_rows_are_not_cut_short(tsa):
    """Scores of 0 over three entries make G exact: bf16(1/3), and bf16(-2/3) at the target.  Rows in the order of their
    targets let the sums of dW climb and come back.  Tensor cores cut a sum at each 16 rows, by 2^-22 of it at most; a
    sum of fp32 that begins anew each 8,192 rows is then off by that of its steps, 2^-24 of the whole for each part
    added, and half a bf16 step in the end."""
    M, V, H = 65536, 3, 128
    h = (1 + torch.rand(M, H, generator=torch.Generator(device=DEV).manual_seed(0), device=DEV)).bfloat16()
    t = torch.arange(M, device=DEV) * V // M
    r = tsa.lm_head_cross_entropy(h, torch.zeros(V, H, dtype=torch.bfloat16, device=DEV), t)
    for v in range(V):
        G = torch.where(t == v, -0.66796875, 0.333984375).double()
        steps = (G[:, None] * h.double()).view(8, 512, 16, H).sum(2)
        want, parts = steps.sum((0, 1)) / M, steps.cumsum(1)
        tol = (2.0 ** -22 * parts.abs().sum((0, 1)) + 8 * U * parts[:, -1].cumsum(0).abs().amax(0)) / M
        near(r.grad_weight[v], want, tol + 2.0 ** -8 * (want.abs() + tol), v)


# of a piece of 30,000 entries each sum of dH takes a third: 10,000 terms, on single CTAs and on pairs
@pytest.mark.parametrize("M,V,H", [(300, 30_000, 4096), (1000, 29_000, 2048)])
def test_sums_of_hidden_gradients_in_several_parts(tsa, M, V, H):
    c = make(M, M, V, H, skip=0.05)
    check(c, tsa.lm_head_cross_entropy(c["h"], c["w"], c["t"]))
