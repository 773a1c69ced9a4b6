"""lm_head_int8 on the GPU against exact integer sums.

Tolerance, with u = 2^-24: the integer sum is exact and rounded once to fp32, two scales and a bias round again:
3 u of the product and u of the result, plus the output's rounding."""
import pytest
import torch

from oracle import head

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DTS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def tsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import top_sampling_apply_gb300 as lib

    lib.load_library()
    return lib


def make(seed, M, V, H, pad=0, fill=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.full((M, H + pad), 113, dtype=torch.int8, device=DEV)[:, :H]
    w = torch.full((V, H + pad), 113, dtype=torch.int8, device=DEV)[:, :H]
    for t in (h, w):
        t.copy_(torch.randint(-128, 128, t.shape, generator=g, device=DEV) if fill is None else
                torch.full(t.shape, fill, device=DEV))
    return dict(h=h, hs=torch.rand(M, generator=g, device=DEV) + 0.01, w=w,
                ws=(torch.rand(V, generator=g, device=DEV) + 0.01) * 1e-4, b=torch.randn(V, generator=g, device=DEV))


def check(c, got, bias):
    s, z = head.int8_scores(c["h"], c["hs"], c["w"], c["ws"], c["b"] if bias else None)
    exact = (s * c["hs"].double()[:, None] * c["ws"].double()).abs()
    f = torch.finfo(got.dtype)
    tol = 3 * U * exact + U * z.abs()
    tol = tol + (0 if got.dtype == torch.float32 else f.eps / 2 * (z.abs() + tol)) + f.smallest_normal * f.eps / 2
    err = (got.double() - z).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 200, 257])
@pytest.mark.parametrize("V,H", [(1, 16), (33, 64), (1000, 80), (4099, 528)])
def test_sizes(tsa, M, V, H):
    c = make(M + V, M, V, H)
    check(c, tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], dtype=torch.float32), False)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("M", [1, 7, 40, 150])
def test_types_bias_strides(tsa, dt, M):
    c = make(M, M, 3001, 336, pad=48)
    for pad in (0, 3):
        buf = torch.full((M, 3001 + pad), float("nan"), dtype=dt, device=DEV)
        got = tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], bias=c["b"], dtype=dt, out=buf[:, :3001])
        check(c, got, True)
        assert torch.isnan(buf[:, 3001:]).all()


@pytest.mark.parametrize("fill", [127, -128])
@pytest.mark.parametrize("M", [1, 40, 130])
@pytest.mark.parametrize("H", [1024, 4112, 16384])
def test_largest_sums_are_exact(tsa, fill, M, H):
    c = make(3, M, 200, H, fill=fill)
    c["h"][0, 5], c["w"][7, H - 1] = 3, -7  # odd sums
    c["hs"].fill_(1.0)
    c["ws"].fill_(1.0)
    got = tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], dtype=torch.float32)
    s, _ = head.int8_scores(c["h"], c["hs"], c["w"], c["ws"])
    assert torch.equal(got, s.float())


def test_scales_that_are_zero_or_not_finite(tsa):
    c = make(1, 5, 300, 64)
    c["hs"][1], c["hs"][2], c["ws"][9] = 0.0, float("nan"), float("nan")
    got = tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], dtype=torch.float32)
    assert (got[1, :9] == 0).all() and torch.isnan(got[2]).all() and torch.isnan(got[:, 9]).all()
    assert torch.isfinite(got[[0, 3, 4]][:, 10:]).all()


@pytest.mark.parametrize("M,H", [(1, 16384), (3, 16384), (10, 5120), (16, 3040), (40, 16384), (130, 8192)])
def test_wide_rows(tsa, M, H):
    c = make(M + H, M, 700, H, pad=32)
    check(c, tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], dtype=torch.float32), False)


def test_large(tsa):
    c = make(2, 300, 50001, 2064)
    check(c, tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"]), False)


def test_scores_of_more_elements_than_32_bits_count(tsa):
    M, V = 17_500, 128_256
    c = make(5, M, V, 64)
    assert M * V > 2 ** 31
    got = tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"])
    last = dict(c, h=c["h"][-300:], hs=c["hs"][-300:])
    check(last, got[-300:], False)


def test_calls_at_once_on_two_streams(tsa):
    cs = [make(30 + i, M, 9000, 1024) for i, M in enumerate((5, 60, 500))]
    want = [tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"]) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_graphs_and_versions(tsa):
    for M in (3, 70):
        c = make(4, M, 2000, 512)
        call = lambda: tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"])  # noqa: E731
        want = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = call()
        torch.cuda.synchronize()
        assert torch.equal(a, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b = call()
        c["h"].copy_(c["h"].flip(0))
        graph.replay()
        assert torch.equal(b, want if M == 1 else call())
    assert tsa.device_status() == 0
    out = torch.empty(70, 2000, dtype=torch.bfloat16, device=DEV)
    tsa.lm_head_int8(c["h"], c["hs"], c["w"], c["ws"], out=out)
    assert out._version == 1
    assert tsa.lm_head_int8(c["h"][:0], c["hs"][:0], c["w"], c["ws"]).shape == (0, 2000)


def test_norm_head_and_draw_together(tsa):
    """The end of a decoding step: the norm in 8 bits, the 8-bit head's scores, a token."""
    g = torch.Generator(device=DEV).manual_seed(0)
    x, r = (torch.randn(12, 256, generator=g, device=DEV).bfloat16() for _ in range(2))
    gain = torch.rand(256, generator=g, device=DEV).bfloat16() + 0.5
    w = torch.randn(2003, 256, generator=g, device=DEV) * 0.2
    wq, ws = tsa.quantize_rows(w)
    n = tsa.rms_norm(x, gain, residual=r, quantize=True)
    z = tsa.lm_head_int8(n.out, n.scale, wq, ws, dtype=torch.float32)
    tokens = tsa.sample(z, 0.0)
    y, _ = head.rms_norm(head.add_residual(x, r), gain, 1e-6)
    want = y @ w.double().T
    # a code is off by half a step on either side (0.501, and a product of the two)
    tol = 0.501 * (n.scale.double()[:, None] * w.double().abs().sum(1) + y.abs().sum(1)[:, None] * ws.double()) \
        + 0.26 * 256 * n.scale.double()[:, None] * ws.double()
    assert ((z.double() - want).abs() <= tol).all()
    assert torch.equal(tokens, z.argmax(-1))
    # and much nearer in the mean than at worst
    assert (z.double() - want).norm() / want.norm() < 0.02


def test_refusals(tsa):
    c = make(1, 4, 64, 32)
    h, hs, w, ws = c["h"], c["hs"], c["w"], c["ws"]
    for call in (lambda: tsa.lm_head_int8(h.float(), hs, w, ws), lambda: tsa.lm_head_int8(h, hs[:2], w, ws),
                 lambda: tsa.lm_head_int8(h, hs, w[:, :16], ws), lambda: tsa.lm_head_int8(h, hs, w, hs),
                 lambda: tsa.lm_head_int8(h, hs, w, ws, dtype=torch.int8),
                 lambda: tsa.lm_head_int8(h, hs, w, ws, out=torch.empty(4, 64, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for n in (24, 8):
        with pytest.raises(tsa.TSAError):
            tsa.lm_head_int8(h[:, :n].contiguous(), hs, w[:, :n].contiguous(), ws)
