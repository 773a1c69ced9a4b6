"""lm_head_logprob on the GPU against float64 scores and the float64 selective log-softmax.

Tolerance: a score is an fp32 sum of exact bf16 products, off by at most H 2^-23 sum_h |h w| (as for the
top-k head), plus 2^-21 max(cap, |z|) for the bias and the cap.  A log-probability is (z_i - m) / T - ln Z: with
every score off by at most d it is off by at most 2 d / T, plus the exponentials' and sums' own rounding
(2^-22 + 60 2^-24 for exponents up to 30, V / 128 2^-24 for a chain of additions, 64 2^-24 for the joins)."""
import numpy as np
import pytest
import torch

import oracle

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


def make(seed, M, V, H, bias=False, mask=False, rowT=False, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    hb = torch.full((M, H + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wb = torch.full((V, H + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    h, w = hb[:, :H], wb[:, :H]
    h.copy_(torch.randn(M, H, generator=g, device=DEV))
    w.copy_(torch.randn(V, H, generator=g, device=DEV) * (3 / H ** 0.5))
    c = dict(h=h, w=w, tok=torch.randint(0, V, (M,), generator=g, device=DEV), b=None, T=1.0, allowed=None)
    if bias:
        c["b"] = torch.randn(V, generator=g, device=DEV)
    if mask:
        c["allowed"] = torch.rand(M, V, generator=g, device=DEV) < 0.5
        c["allowed"][torch.arange(M, device=DEV), c["tok"]] = True
    if rowT:
        c["T"] = torch.rand(M, generator=g, device=DEV) + 0.5
    return c


def bits_of(allowed):
    V = allowed.shape[1]
    a = allowed.cpu().numpy()
    full = np.ones((a.shape[0], (V + 31) // 32 * 32), bool)
    full[:, :V] = a
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)


def check(c, got, cap=0.0):
    h, w = c["h"].double(), c["w"].double()
    z = h @ w.T
    d = h.shape[1] * 2.0 ** -23 * (h.abs() @ w.abs().T).amax(1)
    if c["b"] is not None:
        z = z + c["b"].double()
    d = d + 2.0 ** -21 * torch.clamp(z.abs().amax(1), min=cap)
    if cap > 0:
        z = cap * torch.tanh(z / cap)
    if c["allowed"] is not None:
        z = z.masked_fill(~c["allowed"], -torch.inf)
    T = c["T"].double() if torch.is_tensor(c["T"]) else torch.full((len(z),), float(c["T"]), device=DEV).double()
    T = torch.where(T > 0, T, 1.0)
    y = z / T[:, None]
    tok, V = c["tok"], z.shape[1]
    ok = (tok >= 0) & (tok < V)
    want = y.gather(1, tok.clamp(0, V - 1)[:, None])[:, 0] - torch.logsumexp(y, 1)
    want = torch.where(ok & (y.amax(1) > -torch.inf), want, torch.nan).cpu().numpy()
    tol = (2 * d / T).cpu().numpy() + (4 + 60 + V / 128 + 64) * U + 3 * U * np.abs(np.where(np.isfinite(want), want, 0))
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    f = np.isfinite(want)
    assert np.all(np.abs(got - want)[f] <= tol[f]), np.abs(got - want)[f].max()


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 32, 33, 100, 128, 129, 300])
@pytest.mark.parametrize("V,H", [(1, 8), (33, 64), (1000, 72), (4099, 520)])
def test_sizes(tsa, M, V, H):
    c = make(M * 7 + V, M, V, H)
    check(c, tsa.lm_head_logprob(c["h"], c["w"], c["tok"]))


@pytest.mark.parametrize("M", [3, 20, 90, 260])
@pytest.mark.parametrize("V,H", [(257, 128), (32001, 256)])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_bias_cap_mask_temperature_strides(tsa, M, V, H, cap):
    c = make(M + V, M, V, H, bias=True, mask=True, rowT=True, pad=24)
    got = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"], softcap=cap, temperature=c["T"],
                              bitmask=bits_of(c["allowed"]))
    check(c, got, cap)


@pytest.mark.parametrize("M", [5, 40, 200])
def test_special_rows(tsa, M):
    c = make(M, M, 3001, 192, mask=True)
    c["tok"][0], c["tok"][1] = -1, 3001
    c["allowed"][2] = False
    c["allowed"][3, c["tok"][3]] = False
    c["T"] = 0.0  # as 1
    got = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], temperature=0.0, bitmask=bits_of(c["allowed"]))
    check(c, got)
    assert got[3].item() == float("-inf") and torch.isnan(got[:3]).all()


@pytest.mark.parametrize("M", [4, 30, 140])
def test_scores_far_apart_and_infinite(tsa, M):
    c = make(M, M, 2000, 64, bias=True)
    c["b"][5] = 3e4
    c["b"][6:900] = -3e4
    c["tok"][0] = 5
    check(c, tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"]))
    c["b"][5] = float("inf")
    assert torch.isnan(tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"])).all()
    c["b"][5] = float("nan")  # counts as -inf
    c["tok"][c["tok"] == 5] = 7
    got = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"])
    c["b"][5] = float("-inf")
    check(c, got)


def test_agrees_with_the_oracle_and_repeats(tsa):
    c = make(3, 12, 500, 64)
    a = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], temperature=0.7)
    z = c["h"].double() @ c["w"].double().T
    want = oracle.selective_log_softmax(z.cpu().numpy(), c["tok"].cpu().numpy(), 0.7)
    assert np.allclose(a.cpu().numpy(), want, atol=2e-4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], temperature=0.7)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and tsa.device_status() == 0


def test_more_rows_than_one_pass(tsa):
    c = make(5, 8192 + 77, 600, 64)
    check(c, tsa.lm_head_logprob(c["h"], c["w"], c["tok"]))


def test_large(tsa):
    c = make(6, 700, 50001, 1024, bias=True)
    check(c, tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"], softcap=30.0), 30.0)


def test_refusals(tsa):
    h = torch.zeros(2, 16, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(10, 16, dtype=torch.bfloat16, device=DEV)
    tok = torch.zeros(2, dtype=torch.int64, device=DEV)
    for a in ((h.float(), w, tok), (h, w[:, :8], tok), (h, w, tok.int()), (h, w, tok[:1]), (h.cpu(), w, tok),
              (h.t(), w, tok)):
        with pytest.raises(ValueError):
            tsa.lm_head_logprob(*a)
    with pytest.raises(ValueError):
        tsa.lm_head_logprob(h, w, tok, bias=torch.zeros(9, device=DEV))
    with pytest.raises(tsa.TSAError):
        tsa.lm_head_logprob(h, w, tok, softcap=-1.0)
    with pytest.raises(tsa.TSAError):  # H not a multiple of 8
        tsa.lm_head_logprob(h[:, :12], w[:, :12], tok)
    with pytest.raises(tsa.TSAError):  # a base off the 16-byte grid
        tsa.lm_head_logprob(torch.zeros(40, dtype=torch.bfloat16, device=DEV)[1:33].view(2, 16), w, tok)
    assert tsa.lm_head_logprob(h[:0], w, tok[:0]).shape == (0,)


@pytest.mark.parametrize("cap", [1e-3, 0.5, 8.0, 30.0, 1e3, 1e5, 1e7, 3e38])
@pytest.mark.parametrize("M", [3, 20, 90, 260])
@pytest.mark.parametrize("size", [0.02, 6.0])
def test_soft_caps_of_every_size(tsa, M, cap, size):
    # One column of hidden values 1 and -1: the scores are the weights themselves, without an error of their own.  A
    # capped score is off by 2^-21 of itself (not of the cap), a log-probability by at most twice that, and by the sums'
    # rounding as above.
    g = torch.Generator(device=DEV).manual_seed(M)
    V = 2500
    h, w = torch.zeros(M, 8, device=DEV), torch.zeros(V, 8, device=DEV)
    h[:, 3] = torch.where(torch.arange(M, device=DEV) % 2 == 0, 1.0, -1.0)
    w[:, 3] = torch.randn(V, generator=g, device=DEV) * size
    h, w = h.bfloat16(), w.bfloat16()
    tok = torch.randint(0, V, (M,), generator=g, device=DEV)
    got = tsa.lm_head_logprob(h, w, tok, softcap=cap).double()
    z = h.double() @ w.double().T
    z = cap * torch.tanh(z / cap)
    want = z.gather(1, tok[:, None])[:, 0] - torch.logsumexp(z, 1)
    tol = 2 * 2.0 ** -21 * z.abs().amax(1) + (4 + 60 + V / 128 + 64) * U + 3 * U * want.abs()
    assert torch.all((got - want).abs() <= tol), (got - want).abs().max().item()


def test_soft_cap_of_infinite_scores(tsa):
    # an infinite score is the cap itself; a NaN counts as -inf
    w = torch.zeros(40, 8, device=DEV).bfloat16()
    tok = torch.tensor([0, 1, 2, 5], device=DEV)
    b = torch.zeros(40, device=DEV)
    b[0], b[1], b[2], b[3] = float("inf"), float("-inf"), 2.0, float("nan")
    for M in (4, 40):
        h = torch.zeros(M, 8, device=DEV).bfloat16()
        got = tsa.lm_head_logprob(h, w, tok.repeat(M // 4), bias=b, softcap=4.0).double().cpu().numpy()[:4]
        y = 4.0 * np.tanh(np.array([np.inf, -np.inf, 2.0 / 4.0] + [0.0] * 36))
        want = y[[0, 1, 2, 4]] - np.log(np.exp(y).sum())
        assert np.all(np.abs(got - want) <= 2 * 2.0 ** -21 * 4 + 133 * U), (got, want)


def test_an_output_written_over_is_seen_by_autograd(tsa):
    c = make(1, 5, 100, 64)
    out, x = torch.ones(5, device=DEV), torch.ones(5, device=DEV, requires_grad=True)
    y = (x * out).sum()  # its backward needs out as it was
    assert tsa.lm_head_logprob(c["h"], c["w"], c["tok"], out=out) is out
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        out = torch.ones(5, device=DEV)
    tsa.lm_head_logprob(c["h"], c["w"], c["tok"], out=out)


@pytest.mark.parametrize("M", [3, 20, 40, 128, 129, 300])
@pytest.mark.parametrize("H", [1032, 2056, 5120])
def test_products_of_several_chunks(tsa, M, H):
    # more columns than one sum in the tensor cores takes, and more tiles than SMs
    c = make(M + H, M, 20011, H, bias=True, mask=M == 40 or M == 20, rowT=True)
    got = tsa.lm_head_logprob(c["h"], c["w"], c["tok"], bias=c["b"], softcap=30.0, temperature=c["T"],
                              bitmask=None if c["allowed"] is None else bits_of(c["allowed"]))
    check(c, got, 30.0)


@pytest.mark.parametrize("M,columns", [(3, 512), (20, 512), (40, 1024), (128, 1024), (300, 1024)])
def test_long_sums_are_rounded_outside_the_tensor_cores(tsa, M, columns):
    # Positive products, so that truncation adds up: the score z of token 0 is about 3,000, and the other token's score
    # is 0, so its log-probability is -z.  The tensor cores lose at most an ulp, 2^-23 of their sum, at each step of 16
    # columns, and the sum over a chunk's steps is on average half its end; the chunks' sums are rounded to nearest.
    # (Truncated over all 320 steps z comes out 1.8e-5 of itself too small.)
    H = 5120
    g = torch.Generator(device=DEV).manual_seed(M)
    h = torch.randn(M, H, generator=g, device=DEV).abs().bfloat16()
    w = torch.zeros(2, H, device=DEV)
    w[0] = torch.randn(H, generator=g, device=DEV).abs()
    w = w.bfloat16()
    got = tsa.lm_head_logprob(h, w, torch.ones(M, dtype=torch.int64, device=DEV)).double()
    z = h.double() @ w[0].double()
    steps = columns // 16
    assert torch.all((got + z).abs() <= z * ((steps + 1) / 2 * 2.0 ** -23 + H / columns * U + 3 * U))


@pytest.mark.parametrize("M", [2, 70, 300])
def test_replays_in_a_graph(tsa, M):
    cases = [make(s, M, 3001, 1096, bias=True) for s in (1, 2)]
    a = {k: cases[0][k].clone() for k in ("h", "w", "tok", "b")}
    out = torch.empty(M, device=DEV)

    def run(to=None):
        return tsa.lm_head_logprob(a["h"], a["w"], a["tok"], bias=a["b"], softcap=20.0, out=to)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out)
    for c in cases[::-1]:
        for k in a:
            a[k].copy_(c[k])
        g.replay()
        assert torch.equal(out, run())
